// tk_embedding.hip -- embedding lookup with scaling and dropout, and the table's gradient by
// sorted tokens.
#include "tk_row_checks.h"
#include "tk_rows.h"

namespace tk {

// ---------------------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------------------
struct LookupArgs {
  const void *ids, *table;
  void *y;
  uint64_t row0, ldt, ldy, vocab;
  uint32_t cols, chunks, chunks_per_row;
  Divisor per_row;  // chunks_per_row
  float scale;
  bool ids64;
  Drop drop;
};

// The token of a row; beyond any vocabulary where it is negative.
__device__ __forceinline__ uint64_t token(const void *ids, bool ids64, uint64_t row) {
  return ids64 ? (uint64_t)((const int64_t *)ids)[row] : (uint64_t)(int64_t)((const int32_t *)ids)[row];
}

// A thread takes one chunk: rows come from anywhere in the table, so nothing is gained by keeping a
// row's lanes together, and many waves hide the two loads that wait for each other (the token, then
// its row).
template <class W, class R, bool kDivide, int CH>
__global__ __launch_bounds__(256) void k_embedding(LookupArgs a) {
  const uint32_t n = blockIdx.x * 256u + threadIdx.x;
  if (n >= a.chunks) return;
  const uint32_t r = a.per_row.of(n), c = (n - r * a.chunks_per_row) * CH;
  const uint64_t row = a.row0 + r, id = token(a.ids, a.ids64, row);
  const int nv = (int)(a.cols - c);
  float v[CH];
  if (id < a.vocab) {
    unpack<CH, W>(load_chunk<false, CH>((const W *)a.table + id * a.ldt + chunk_at<CH>(c, a.cols)), nv, v);
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] *= a.scale;
    if (a.drop.on) drop_chunk<kDivide, CH>(a.drop, a.drop.start + (uint32_t)row * a.cols + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] = 0.0f;
  }
  store_chunk<CH>((R *)a.y + row * a.ldy + c, nv, v);
}

// ---------------------------------------------------------------------------------------
// The rows in the order of their tokens
// ---------------------------------------------------------------------------------------
struct SortArgs {
  const void *ids;
  uint32_t *order;  // the rows with a token, by token and then by row
  uint32_t *first;  // where each token's rows begin in `order`, and at [vocab] where they end
  uint32_t rows, vocab, ranges;
  bool ids64;
};

constexpr uint32_t kNoToken = ~0u;
constexpr int kSortWaves = 16, kAhead = 8;

// A work-group takes a range of kRange tokens and reads all rows' tokens, which lie in the L2s:
// it needs nothing from the other ones, since the rows of lower tokens that it passes say where its
// own begin.  Each wave reads a sixteenth of the rows, in their order, twice: it counts its tokens
// in a column of its own, and after a scan over tokens and waves it puts its rows in their places.
// Rows of one token keep their order, whatever the waves do, so a gradient's sum has one order.
template <int kRange>
__global__ __launch_bounds__(64 * kSortWaves) void k_sort_tokens(SortArgs a) {
  __shared__ uint32_t count[kSortWaves][kRange], part[kSortWaves], under[kSortWaves];
  const uint32_t lane = threadIdx.x & 63, wave = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t piece = ((a.rows + kSortWaves * 64 - 1) / (kSortWaves * 64)) * 64;
  const uint32_t begin = wave * piece, end = begin + piece < a.rows ? begin + piece : a.rows;
  const auto load = [&](uint32_t i) -> uint32_t {  // the token of row i, or none
    if (i >= end) return kNoToken;
    const uint64_t id = token(a.ids, a.ids64, i);
    return id < a.vocab ? (uint32_t)id : kNoToken;
  };
  for (uint32_t range = blockIdx.x; range < a.ranges; range += gridDim.x) {
    const uint32_t lo = range * kRange;
    for (uint32_t i = threadIdx.x; i < kSortWaves * kRange; i += 64 * kSortWaves) (&count[0][0])[i] = 0;
    __syncthreads();
    uint32_t below = 0;
    for (uint32_t at = begin; at < end; at += 64 * kAhead) {
      uint32_t t[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) t[k] = load(at + 64 * k + lane);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        below += t[k] < lo;
        if (t[k] - lo < kRange) atomicAdd(&count[wave][t[k] - lo], 1u);
      }
    }
    for (int d = 1; d < 64; d <<= 1) below += __shfl_xor(below, d);
    if (lane == 0) under[wave] = below;
    __syncthreads();
    // Where each token's rows begin: a scan over the range's tokens, and within a token over the waves.
    uint32_t total = 0, base = 0;
    if (threadIdx.x < kRange)
      for (int w = 0; w < kSortWaves; ++w) total += count[w][threadIdx.x];
    uint32_t upto = total;
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = __shfl_up(upto, d);
      upto += lane >= (uint32_t)d ? o : 0;
    }
    if (lane == 63) part[wave] = upto;
    __syncthreads();
    for (int w = 0; w < kSortWaves; ++w) base += under[w] + (w < (int)wave ? part[w] : 0);
    if (threadIdx.x < kRange) {
      uint32_t at = base + upto - total;
      if (lo + threadIdx.x < a.vocab) a.first[lo + threadIdx.x] = at;
      if (lo + threadIdx.x + 1 == a.vocab) a.first[a.vocab] = at + total;
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t n = count[w][threadIdx.x];
        count[w][threadIdx.x] = at;
        at += n;
      }
    }
    __syncthreads();
    for (uint32_t at = begin; at < end; at += 64 * kAhead) {
      uint32_t t[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) t[k] = load(at + 64 * k + lane);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        uint64_t left = __ballot(t[k] - lo < kRange);
        while (left) {  // the rows of one token at a time, the first lane's
          const int leader = __ffsll((unsigned long long)left) - 1;
          const uint32_t mine = (uint32_t)__builtin_amdgcn_readlane((int)t[k], leader);
          const uint64_t same = __ballot(t[k] == mine);
          uint32_t put = 0;
          if (lane == (uint32_t)leader) put = atomicAdd(&count[wave][mine - lo], (uint32_t)__popcll(same));
          put = (uint32_t)__builtin_amdgcn_readlane((int)put, leader);
          if (t[k] == mine) a.order[put + __popcll(same & ((1ull << lane) - 1))] = at + 64 * k + lane;
          left &= ~same;
        }
      }
    }
    __syncthreads();  // the next range clears the counts
  }
}

// ---------------------------------------------------------------------------------------
// The gradient
// ---------------------------------------------------------------------------------------
struct GradArgs {
  const void *ids, *dy;
  const uint32_t *order, *first;
  void *dtable;
  float *partial;  // two lines to a tile of `order`
  uint64_t lddy, lddt;
  uint32_t rows, vocab, cols, tile, tiles, strips, hot_groups;
  float scale;
  bool ids64;
  Drop drop;
};

// A token of up to `tile` rows is summed by the group of lanes that writes its gradient.  Of one with
// more, its parts between the multiples of `tile` in `order` are summed by a group each, to a line of
// the workspace, and k_join adds the lines: a text's most frequent token has a tenth of the rows.
// A tile holds at most two such parts: of a token that begins before it (its first line) and of one
// that begins in it (its second).
template <class W, class R, bool kDivide, bool kAdd, int CH, int kLanes>
struct Sums {
  const GradArgs &a;
  uint32_t c, lane;  // this lane's first column, and its place in the group
  int nv;

  // drop(dy) of the rows order[from .. to), added up in that order
  __device__ __forceinline__ void rows(uint32_t from, uint32_t to, float *acc) const {
    constexpr int kDeep = 4;
#pragma unroll
    for (int e = 0; e < CH; ++e) acc[e] = 0.0f;
    const uint32_t at = chunk_at<CH>(c, a.cols);
    for (uint32_t i = from; i < to; i += kDeep) {
      Chunk<R, CH> x[kDeep];
      uint32_t r[kDeep];
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        r[k] = a.order[i + k < to ? i + k : to - 1];
        if (kLanes == 64) r[k] = (uint32_t)__builtin_amdgcn_readfirstlane(r[k]);
      }
#pragma unroll
      for (int k = 0; k < kDeep; ++k)
        if (i + k < to) x[k] = load_chunk<false, CH>((const R *)a.dy + r[k] * a.lddy + at);
#pragma unroll
      for (int k = 0; k < kDeep; ++k)
        if (i + k < to) {
          float v[CH];
          unpack<CH, R>(x[k], nv, v);
          if (a.drop.on) drop_chunk<kDivide, CH>(a.drop, a.drop.start + r[k] * a.cols + c, v);
#pragma unroll
          for (int e = 0; e < CH; ++e) acc[e] += v[e];
        }
    }
  }
  __device__ __forceinline__ void write(uint32_t id, float *acc) const {
    W *p = (W *)a.dtable + id * a.lddt;
#pragma unroll
    for (int e = 0; e < CH; ++e) acc[e] *= a.scale;
    if (kAdd) {
      float old[CH];
      unpack<CH, W>(load_chunk<false, CH>(p + chunk_at<CH>(c, a.cols)), nv, old);
#pragma unroll
      for (int e = 0; e < CH; ++e) acc[e] += old[e];
    }
    store_chunk<CH>(p + c, nv, acc);
  }
  // One of the vocabulary's tokens, or (adding to what is there) the token that begins at a place
  // of `order`, so that nothing is looked up for the tokens that do not occur.
  __device__ __forceinline__ void cold(uint32_t n) const {
    uint32_t id = n;
    if (kAdd) {
      if (n >= a.first[a.vocab]) return;
      id = (uint32_t)token(a.ids, a.ids64, a.order[n]);
    }
    const uint32_t s = a.rows ? a.first[id] : 0, e = a.rows ? a.first[id + 1] : 0;
    if (e - s > a.tile || (kAdd && s != n)) return;
    float acc[CH];
    rows(s, e, acc);
    write(id, acc);
  }
  __device__ __forceinline__ void hot(uint32_t t) const {
    const uint32_t all = a.first[a.vocab], from = t * a.tile;
    if (from >= all) return;
    const uint32_t to = all - from < a.tile ? all : from + a.tile;
    float acc[CH];
    const auto part = [&](uint32_t id, int line) {
      const uint32_t s = a.first[id], e = a.first[id + 1];
      if (e - s <= a.tile || (s < from) != (line == 0)) return;
      rows(s < from ? from : s, e < to ? e : to, acc);
      put_sums<CH>(a.partial + (2ull * t + line) * line_pitch(a.cols) + c, nv, acc);
    };
    part((uint32_t)token(a.ids, a.ids64, a.order[from]), 0);
    part((uint32_t)token(a.ids, a.ids64, a.order[to - 1]), 1);
  }
};

template <class W, class R, bool kDivide, bool kAdd, int CH, int kLanes>
__global__ __launch_bounds__(256) void k_token_sums(GradArgs a) {
  constexpr uint32_t kGroups = 256 / kLanes;
  uint32_t group = threadIdx.x / kLanes;
  if (kLanes == 64) group = (uint32_t)__builtin_amdgcn_readfirstlane(group);
  const uint32_t lane = threadIdx.x % kLanes, units = kAdd ? a.rows : a.vocab, groups = (units + kGroups - 1) / kGroups;
  for (uint32_t strip = blockIdx.x; strip < a.strips; strip += gridDim.x) {
    const uint32_t c = (strip * kLanes + lane) * CH;
    if (c >= a.cols) continue;
    const Sums<W, R, kDivide, kAdd, CH, kLanes> sums{a, c, lane, (int)(a.cols - c)};
    for (uint32_t g = blockIdx.y; g < a.hot_groups + groups; g += gridDim.y) {
      if (g < a.hot_groups) {
        const uint32_t t = g * kGroups + group;
        if (t < a.tiles) sums.hot(t);
      } else {
        const uint32_t n = (g - a.hot_groups) * kGroups + group;
        if (n < units) sums.cold(n);
      }
    }
  }
}

// The tokens of more than `tile` rows: their lines, in order.  blockIdx.y: the tile where one begins.
template <class W, bool kAdd>
__global__ __launch_bounds__(256) void k_join(GradArgs a) {
  const uint32_t all = a.first[a.vocab], t = blockIdx.y, from = t * a.tile;
  if (from >= all) return;
  const uint32_t to = all - from < a.tile ? all : from + a.tile;
  const uint32_t id = (uint32_t)token(a.ids, a.ids64, a.order[to - 1]), s = a.first[id], e = a.first[id + 1];
  if (e - s <= a.tile || s < from) return;
  const uint64_t pitch = line_pitch(a.cols);
  const uint32_t last = (e - 1) / a.tile;
  for (uint64_t c = blockIdx.x * 256ull + threadIdx.x; c < a.cols; c += gridDim.x * 256ull) {
    const float *p = a.partial + 2ull * t * pitch + c;
    float sum = p[pitch];
    for (uint32_t k = t + 1; k <= last; k += 8) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = p[2ull * ((k + j < last ? k + j : last) - t) * pitch];
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += k + j <= last ? v[j] : 0.0f;
    }
    W *out = (W *)a.dtable + id * a.lddt + c;
    sum *= a.scale;
    *out = (W)(kAdd ? sum + (float)*out : sum);
  }
}

// ---------------------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------------------
// Rows of `order` to a tile: 64, and more where that makes over 1024 tiles.
constexpr uint64_t kLeastTile = 64, kMostTiles = 1024;

static uint32_t tile_of(uint64_t rows) {
  uint64_t t = kLeastTile;
  while ((rows + t - 1) / t > kMostTiles) t *= 2;
  return (uint32_t)t;
}

static uint64_t most_tiles(uint64_t rows) {
  const uint64_t t = (rows + kLeastTile - 1) / kLeastTile;
  return rows <= kLeastTile ? 0 : t < kMostTiles ? t : kMostTiles;  // a single tile has no token of more rows
}

static uint64_t embedding_bytes(uint64_t rows, uint64_t cols, uint64_t vocab) {
  if (rows == 0 || cols == 0 || vocab == 0) return 0;
  return 4 * (rows + vocab + 1) + 8 * most_tiles(rows) * line_pitch(cols) + 12;  // 12: the lines are aligned to 16 bytes
}

template <class W, class R, bool kDivide>
struct Embedding {
  static constexpr int CH = kChunk<W, R>;

  static tk_status forward(LookupArgs a, uint64_t rows, hipStream_t s) {
    const int ch = a.cols < (uint32_t)CH ? 1 : CH;
    a.chunks_per_row = (a.cols + ch - 1) / ch;
    a.per_row = Divisor(a.chunks_per_row);
    const uint64_t rows_each = (1ull << 30) / a.chunks_per_row;
    for (uint64_t r = 0; r < rows; r += rows_each) {
      a.row0 = r;
      a.chunks = (uint32_t)((rows - r < rows_each ? rows - r : rows_each) * a.chunks_per_row);
      const dim3 grid((a.chunks + 255) / 256);
      if (ch == 1) hipLaunchKernelGGL((k_embedding<W, R, kDivide, 1>), grid, dim3(256), 0, s, a);
      else hipLaunchKernelGGL((k_embedding<W, R, kDivide, CH>), grid, dim3(256), 0, s, a);
      const tk_status st = launch_status();
      if (st != TK_OK) return st;
    }
    return TK_OK;
  }

  template <bool kAdd, int ch, int kLanes>
  static void launch_sums(GradArgs a, hipStream_t s) {
    constexpr uint32_t kGroups = 256 / kLanes;
    const uint64_t units = kAdd ? a.rows : a.vocab, groups = (units + kGroups - 1) / kGroups;
    a.strips = (uint32_t)(((uint64_t)a.cols + kLanes * ch - 1) / (kLanes * ch));
    a.hot_groups = (a.tiles + kGroups - 1) / kGroups;
    const uint64_t g = a.hot_groups + groups;
    hipLaunchKernelGGL((k_token_sums<W, R, kDivide, kAdd, ch, kLanes>),
                       dim3(a.strips < 1u << 16 ? a.strips : 1u << 16, (uint32_t)(g < 32768 ? g : 32768)), dim3(256), 0, s, a);
  }
  template <bool kAdd>
  static tk_status sums(const GradArgs &a, hipStream_t s) {
    if (a.cols < (uint32_t)CH) launch_sums<kAdd, 1, 8>(a, s);
    else if (a.cols <= 8u * CH) launch_sums<kAdd, CH, 8>(a, s);
    else if (a.cols <= 16u * CH) launch_sums<kAdd, CH, 16>(a, s);
    else if (a.cols <= 32u * CH) launch_sums<kAdd, CH, 32>(a, s);
    else launch_sums<kAdd, CH, 64>(a, s);
    tk_status st = launch_status();
    if (st != TK_OK || a.tiles == 0) return st;
    const uint32_t blocks = (a.cols + 255) / 256;
    hipLaunchKernelGGL((k_join<W, kAdd>), dim3(blocks < 1024 ? blocks : 1024, a.tiles), dim3(256), 0, s, a);
    return launch_status();
  }
  static tk_status backward(const GradArgs &a, bool add, hipStream_t s) { return add ? sums<true>(a, s) : sums<false>(a, s); }
};

static tk_status sort_tokens(SortArgs a, hipStream_t s) {
  const auto go = [&](auto kernel, uint32_t range) {
    a.ranges = (a.vocab + range - 1) / range;
    hipLaunchKernelGGL(kernel, dim3(a.ranges < 1u << 16 ? a.ranges : 1u << 16), dim3(64 * kSortWaves), 0, s, a);
  };
  // one work-group to a compute unit where the vocabulary allows: each reads all rows
  if (a.vocab <= 64 * 256) go(k_sort_tokens<64>, 64);
  else if (a.vocab <= 128 * 256) go(k_sort_tokens<128>, 128);
  else if (a.vocab <= 256 * 256) go(k_sort_tokens<256>, 256);
  else go(k_sort_tokens<512>, 512);
  return launch_status();
}

// Calls f with the kernels of a call's types.
template <class F>
static tk_status with_types(RowType t, uint32_t flags, F f) {
  const bool r32 = flags & TK_RESIDUAL_F32, w32 = flags & TK_PARAMS_F32;
  const auto half = [&](auto h) {
    typedef decltype(h) H;
    if (w32) return r32 ? f(Embedding<float, float, false>()) : f(Embedding<float, H, false>());
    return r32 ? f(Embedding<H, float, false>()) : f(Embedding<H, H, false>());
  };
  switch (t) {
    case kF16: return half(f16_t());
    case kBF16: return half(bf16_t());
    default: return f(Embedding<float, float, true>());
  }
}

static tk_status check_lookup(uint64_t start, uint64_t rows, uint64_t cols, float p, float scale, uint32_t flags,
                              uint32_t allowed, uint64_t vocab) {
  if (!(scale > -INFINITY && scale < INFINITY)) return TK_EINVAL;
  const tk_status st = check_scalars(start, rows, cols, p, 0.0f, flags, allowed);
  return st != TK_OK ? st : vocab >= kMaxDim ? TK_ERANGE : TK_OK;
}

constexpr uint32_t kLookupFlags = TK_RESIDUAL_F32 | TK_PARAMS_F32 | TK_INDEX_I64;
constexpr int kTable = 2;  // Region's kind: rows of the table, which no other matrix may be

static tk_status embedding(RowType t, uint32_t key, uint64_t start, uint64_t rows, uint64_t cols, float p, float scale,
                           uint32_t flags, uint64_t vocab, const void *ids, const void *table, uint64_t ldt, void *y,
                           uint64_t ldy, hipStream_t stream) {
  tk_status st = check_lookup(start, rows, cols, p, scale, flags, kLookupFlags, vocab);
  if (st != TK_OK || rows == 0 || cols == 0) return st;
  Arguments c{t, rows, cols, flags};
  c.vector(ids, rows, flags & TK_INDEX_I64 ? 8 : 4, false, true);
  if (vocab) c.matrix_of(table, vocab, cols, ldt, c.par(), false, true, kTable);
  c.matrix(y, ldy, c.res(), true, true);
  if ((st = c.done()) != TK_OK) return st;
  LookupArgs a{};
  a.ids = ids; a.ids64 = flags & TK_INDEX_I64; a.table = table; a.ldt = ldt; a.y = y; a.ldy = ldy;
  a.vocab = vocab; a.cols = (uint32_t)cols; a.scale = scale;
  a.drop = drop_of(key, start, p);
  return with_types(t, flags, [&](auto k) { return k.forward(a, rows, stream); });
}

static tk_status embedding_backward(RowType t, uint32_t key, uint64_t start, uint64_t rows, uint64_t cols, float p,
                                    float scale, uint32_t flags, uint64_t vocab, const void *ids, const void *dy,
                                    uint64_t lddy, void *dtable, uint64_t lddt, void *workspace, uint64_t bytes,
                                    hipStream_t stream) {
  tk_status st = check_lookup(start, rows, cols, p, scale, flags, kLookupFlags | TK_ACCUMULATE, vocab);
  const bool add = flags & TK_ACCUMULATE;
  if (st != TK_OK || cols == 0 || vocab == 0 || (rows == 0 && add)) return st;
  Arguments c{t, rows, cols, flags};
  if (rows) {
    c.vector(ids, rows, flags & TK_INDEX_I64 ? 8 : 4, false, true);
    c.matrix(dy, lddy, c.res(), false, true);
  }
  c.matrix_of(dtable, vocab, cols, lddt, c.par(), true, true, kTable);
  const uint64_t need = embedding_bytes(rows, cols, vocab);
  if (!serves(workspace, bytes, need)) return TK_EINVAL;
  if (need) c.vector(workspace, need / 4, 4, true, true);
  if ((st = c.done()) != TK_OK) return st;
  GradArgs a{};
  a.ids = ids; a.ids64 = flags & TK_INDEX_I64; a.dy = dy; a.lddy = lddy; a.dtable = dtable; a.lddt = lddt;
  a.rows = (uint32_t)rows; a.vocab = (uint32_t)vocab; a.cols = (uint32_t)cols; a.scale = scale;
  a.drop = drop_of(key, start, p);
  if (rows) {
    uint32_t *order = (uint32_t *)workspace, *first = order + rows;
    a.order = order;
    a.first = first;
    a.partial = (float *)(((uintptr_t)(first + vocab + 1) + 15) & ~(uintptr_t)15);
    a.tile = tile_of(rows);
    a.tiles = rows <= a.tile ? 0 : (uint32_t)((rows + a.tile - 1) / a.tile);
    if ((st = sort_tokens(SortArgs{ids, order, first, a.rows, a.vocab, 0, a.ids64}, stream)) != TK_OK) return st;
  }
  return with_types(t, flags, [&](auto k) { return k.backward(a, add, stream); });
}

}  // namespace tk

extern "C" {

tk_status tk_embedding_workspace_bytes(uint64_t rows, uint64_t cols, uint64_t vocab, uint64_t *bytes) {
  if (!bytes) return TK_EINVAL;
  if (rows >= tk::kMaxDim || cols >= tk::kMaxDim || vocab >= tk::kMaxDim) return TK_ERANGE;
  *bytes = tk::embedding_bytes(rows, cols, vocab);
  return TK_OK;
}

#define TK_EMBEDDING(SUFFIX, TYPE)                                                                                        \
  tk_status tk_embedding_##SUFFIX(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p, float scale,  \
                                  uint32_t flags, uint64_t vocab, const void *ids, const void *table, uint64_t ldt,       \
                                  void *y, uint64_t ldy, hipStream_t stream) {                                            \
    return tk::embedding(TYPE, key, start_draw, rows, cols, p, scale, flags, vocab, ids, table, ldt, y, ldy, stream);     \
  }                                                                                                                       \
  tk_status tk_embedding_backward_##SUFFIX(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p,      \
                                           float scale, uint32_t flags, uint64_t vocab, const void *ids, const void *dy,  \
                                           uint64_t lddy, void *dtable, uint64_t lddt, void *workspace,                   \
                                           uint64_t workspace_bytes, hipStream_t stream) {                                \
    return tk::embedding_backward(TYPE, key, start_draw, rows, cols, p, scale, flags, vocab, ids, dy, lddy, dtable, lddt, \
                                  workspace, workspace_bytes, stream);                                                    \
  }

TK_EMBEDDING(f32, tk::kF32)
TK_EMBEDDING(f16, tk::kF16)
TK_EMBEDDING(bf16, tk::kBF16)

}  // extern "C"
