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

// Bound by memory: bf16 16384x4096 from a table of 131072 rows, with dropout, 47 us, 5.5 TB/s (one chunk to a
// lane 50, four 49; a row's address made by every lane for itself 58).
//
// A lane takes V chunks, 64 apart.  Rows come from anywhere in the table, so nothing is gained by going
// on from one to the next: many waves hide the two loads that wait for each other (the token, then its
// row).  kWide: a wave takes 64 V chunks of one row, whose token and address are the scalar unit's; else
// (V = 1) the chunks of all rows follow each other.  From 64 chunks on, which gains on long rows and loses where
// the row's last wave has many lanes idle.  us, wide and chunk by chunk, 2^25 elements from a table of 32768 rows:
//      columns              512       1024       1152       1536       2048       4096
//      bf16              22.9 20.6  21.0 20.7  23.8 20.9  22.3 20.9  21.3 21.0  21.4 21.0 (16384x4096 of 131072: 47.5 55.9)
//      bf16, dropout     31.3 22.6  22.2 22.1  28.3 22.5  23.7 22.3  22.2 22.3  22.5 22.2
//      f32               39.2 38.7  39.4 38.8  40.2 39.2  39.6 39.1  39.8 39.0  40.8 44.4
template <class W, class R, bool kDivide, int CH, bool kWide, int V>
__global__ __launch_bounds__(256) void k_embedding(LookupArgs a) {
  uint32_t n, r, c;
  if constexpr (kWide) {
    n = blockIdx.x * 4u + (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (n >= a.chunks) return;  // here waves' worth of chunks
    r = a.per_row.of(n);
    c = ((n - r * a.chunks_per_row) * (64 * V) + (threadIdx.x & 63)) * CH;
  } else {
    n = blockIdx.x * 256u + threadIdx.x;
    if (n >= a.chunks) return;
    r = a.per_row.of(n);
    c = (n - r * a.chunks_per_row) * CH;
  }
  const uint64_t row = a.row0 + r, id = token(a.ids, a.ids64, row);
  const bool there = id < a.vocab;
  Chunk<W, CH> x[V];
  if (there)
#pragma unroll
    for (int j = 0; j < V; ++j)
      x[j] = load_chunk<false, CH>((const W *)a.table + id * a.ldt + chunk_at<CH>(c + j * 64 * CH, a.cols));
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t at = c + j * 64 * CH;
    const int nv = (int)(a.cols - at);
    float v[CH];
    if (there) {
      unpack<CH, W>(x[j], nv, v);
#pragma unroll
      for (int e = 0; e < CH; ++e) v[e] *= a.scale;
      if (a.drop.on) {
        if constexpr (CH > 1) {
          uint32_t w[CH];
          chunk_words<CH>(a.drop.hk, a.drop.start + (uint32_t)row * a.cols + at, w);
#pragma unroll
          for (int e = 0; e < CH; ++e) v[e] = drop_one<kDivide>(a.drop, w[e], v[e]);
        } else {
          drop_chunk<kDivide, CH>(a.drop, a.drop.start + (uint32_t)row * a.cols + at, v);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < CH; ++e) v[e] = 0.0f;
    }
    if (nv > 0) store_chunk<CH>((R *)a.y + row * a.ldy + at, nv, v);
  }
}

// ---------------------------------------------------------------------------------------
// The rows in the order of their tokens
// ---------------------------------------------------------------------------------------
struct SortArgs {
  const void *ids;
  uint32_t *order;  // the rows with a token, by token and then by row
  uint32_t *run;    // at a token's first place in `order` the number of its rows, else 0
  uint32_t *first;  // where each token's rows begin in `order`, and at [vocab] where they end
  uint32_t rows, vocab, ranges;
  bool ids64;
};

constexpr uint32_t kNoToken = ~0u;
constexpr int kSortWaves = 16, kAhead = 8;

// The lanes whose number below kRange is this lane's, among those of `mask`: a vote for each bit.
template <int kRange>
__device__ __forceinline__ uint64_t same_lanes(uint32_t n, uint64_t mask) {
  uint32_t lo = (uint32_t)mask, hi = (uint32_t)(mask >> 32);
#pragma unroll
  for (int b = 0; (1 << b) < kRange; ++b) {
    const uint64_t set = __ballot((n >> b) & 1);
    const uint32_t mine = (uint32_t)((int)(n << (31 - b)) >> 31);  // this lane's bit in all of them
    lo &= ~((uint32_t)set ^ mine);
    hi &= ~((uint32_t)(set >> 32) ^ mine);
  }
  return (uint64_t)hi << 32 | lo;
}

// Counts that a wave's lanes read and its first lanes of each token write, in this order: a wave's LDS
// accesses are not reordered.
__device__ __forceinline__ uint32_t get_count(uint32_t *p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
}
__device__ __forceinline__ void set_count(uint32_t *p, uint32_t n) {
  __hip_atomic_store(p, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
}

// A work-group takes a range of kRange tokens and reads all rows' tokens, which lie in the L2s:
// it needs nothing from the other ones, since the rows of lower tokens that it passes say where its
// own begin.  Each wave reads a sixteenth of the rows, in their order, twice: it counts its tokens
// in a column of its own, and after a scan over tokens and waves it puts its rows in their places.
// Rows of one token keep their order, whatever the waves do, so a gradient's sum has one order.
//
// Bound by two passes over all rows' tokens in every work-group, whatever the tokens are, and beyond that by
// the work-group that has the most rows of its own: of a text's tokens half are among the lowest hundred.
// us, rows evenly spread, text-like, and all one token's:
//                       4096 rows        16384 rows         65536 rows
//      32768 tokens   7.3  7.7  9.9    12.0 15.2 26.1    27.4 48.2 93.1
//     131072 tokens                    12.4 16.6 27.7    29.5 54.5 98.6
// The lanes of one token find each other by votes, and the first of them moves its place on for all (with a
// turn of a loop for each of a wave's tokens the 15.2 us are 82).  Counted by votes as well, so that the second
// pass has no more to do, they are 17, and the 26 are 14, where the counts wait for each other.
template <int kRange, bool kI64>
__global__ __launch_bounds__(64 * kSortWaves) void k_sort_tokens(SortArgs a) {
  __shared__ uint32_t count[kSortWaves][kRange], begin_of[kRange], total_of[kRange], part[kSortWaves], under[kSortWaves];
  const uint32_t lane = threadIdx.x & 63, wave = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t under_me = (1ull << lane) - 1;
  const uint32_t piece = ((a.rows + kSortWaves * 64 - 1) / (kSortWaves * 64)) * 64;
  const uint32_t begin = wave * piece, end = begin + piece < a.rows ? begin + piece : a.rows;
  // The token of row i, or none.  Loaded in any case: loads in branches wait for each other.
  const auto load = [&](uint32_t i) -> uint32_t {
    const uint64_t id = token(a.ids, kI64, i < a.rows ? i : a.rows - 1);
    return (i < end) & (id < a.vocab) ? (uint32_t)id : kNoToken;  // no branch
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
      begin_of[threadIdx.x] = at;
      total_of[threadIdx.x] = total;
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
        const uint32_t own = t[k] - lo;
        const uint64_t mine = __ballot(own < kRange);
        if (mine) {
          const uint64_t same = same_lanes<kRange>(own, mine);
          if (own < kRange) {
            const uint32_t put = get_count(&count[wave][own]), place = put + (uint32_t)__popcll(same & under_me);
            if ((same & under_me) == 0) set_count(&count[wave][own], put + (uint32_t)__popcll(same));
            a.order[place] = at + 64 * k + lane;
            a.run[place] = place == begin_of[own] ? total_of[own] : 0;
          }
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
  const uint32_t *order, *run, *first;
  void *dtable;
  float *partial;  // two lines to a tile of `order`
  uint64_t lddy, lddt, units, strips, blocks;  // units: tiles times strips; blocks: work-groups' worth of work
  uint32_t rows, vocab, cols, tile, tiles;
  uint32_t clear_lanes;  // lanes that clear a row whose token does not occur (0: none are cleared)
  float scale;
  bool ids64;
  Drop drop;
};

// A group of lanes takes a tile, `tile` places of `order` after each other, and a strip of columns: all
// have the same work, whether a text's most frequent token has a tenth of the rows or every row has
// a token of its own.  It reads the rows ahead of adding them, and where a token ends writes its
// gradient.  Of a token that goes past an end of the tile it writes the sum so far, to a line of the
// workspace: the tile's first line if the token begins before the tile, else its second.  k_join adds
// those lines up in the order of the tiles.
//
// Bound by memory: bf16 16384x4096 into a table of 32768 rows, text-like tokens, 68 us with the rows that are
// cleared, 6.0 TB/s of the 409 MB that the counters show (with eight rows ahead, at fewer waves, 72; with a wave
// to each token and strip 128).
template <class W, class R, bool kDivide, bool kAdd, int CH, int kLanes>
struct Tile {
  static constexpr int kDeep = 4;
  const GradArgs &a;
  uint32_t c, lane;  // this lane's first column, and its place in the group
  int nv;

  // A value that the lane of place i holds.
  __device__ __forceinline__ uint32_t of_place(uint32_t v, uint32_t i) const {
    return kLanes == 64 ? (uint32_t)__builtin_amdgcn_readlane((int)v, (int)i) : (uint32_t)__shfl((int)v, (int)i, kLanes);
  }
  __device__ __forceinline__ Chunk<R, CH> load(uint32_t row) const {
    return load_chunk<false, CH>((const R *)a.dy + row * a.lddy + chunk_at<CH>(c, a.cols));
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
  __device__ __forceinline__ void put_line(uint32_t t, int line, const float *acc) const {
    put_sums<CH>(a.partial + (2ull * t + line) * line_pitch(a.cols) + c, nv, acc);
  }
  __device__ __forceinline__ void run(uint32_t t) const {
    const uint32_t all = a.first[a.vocab], t0 = t * a.tile;
    if (t0 >= all) return;
    const uint32_t n = all - t0 < a.tile ? all - t0 : a.tile, place = t0 + (lane < n ? lane : n - 1);
    const uint32_t row = a.order[place];
    const bool ends = place + 1 == all || a.run[place + 1] != 0;
    bool whole = a.run[t0] != 0;  // the token began in this tile
    const uint32_t id = (uint32_t)token(a.ids, a.ids64, row);
    const uint64_t end_mask = __ballot(ends);
    Chunk<R, CH> x[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k)
      if ((uint32_t)k < n) x[k] = load(of_place(row, k));
    float acc[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) acc[e] = 0.0f;
    for (uint32_t i0 = 0; i0 < n; i0 += kDeep) {
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const uint32_t i = i0 + k;
        if (i >= n) break;
        float v[CH];
        unpack<CH, R>(x[k], nv, v);
        if (i + kDeep < n) x[k] = load(of_place(row, i + kDeep));
        if (a.drop.on) drop_chunk<kDivide, CH>(a.drop, a.drop.start + of_place(row, i) * a.cols + c, v);
#pragma unroll
        for (int e = 0; e < CH; ++e) acc[e] += v[e];
        const bool end = kLanes == 64 ? (end_mask >> i) & 1 : of_place(ends, i) != 0;
        if (!end) continue;
        if (whole) write(of_place(id, i), acc);
        else put_line(t, 0, acc);
        whole = true;
#pragma unroll
        for (int e = 0; e < CH; ++e) acc[e] = 0.0f;
      }
    }
    if (!(kLanes == 64 ? (end_mask >> (n - 1)) & 1 : of_place(ends, n - 1) != 0)) put_line(t, whole ? 1 : 0, acc);
  }
};

// `lanes` lanes clear n bytes, whole elements of `size`: vectors between the 16-byte boundaries.
__device__ __forceinline__ void clear_row(char *p, uint64_t n, uint32_t size, uint32_t lane, uint32_t lanes) {
  typedef uint32_t V4 __attribute__((ext_vector_type(4)));
  uint64_t head = (16 - ((uintptr_t)p & 15)) & 15;
  head = head < n ? head : n;
  const uint64_t vectors = (n - head) / 16, tail = head + vectors * 16;
  const auto one = [&](uint64_t at) {
    if (size == 4) *(uint32_t *)(p + at) = 0;
    else *(uint16_t *)(p + at) = 0;
  };
  if (lane * size < head) one(lane * size);
  if (tail + lane * size < n) one(tail + lane * size);
  for (uint64_t i = lane; i < vectors; i += lanes) __builtin_nontemporal_store(V4(0), (V4 *)(p + head) + i);
}

// Work-groups of four waves.  The tiles come first: the rows to clear, whose stores wait for nothing,
// fill the time that the tiles wait for their loads.
template <class W, class R, bool kDivide, bool kAdd, int CH, int kLanes>
__global__ __launch_bounds__(256) void k_token_sums(GradArgs a) {
  constexpr uint32_t kGroups = 256 / kLanes;
  uint32_t group = threadIdx.x / kLanes;
  if (kLanes == 64) group = (uint32_t)__builtin_amdgcn_readfirstlane(group);
  const uint64_t sums = (a.units + kGroups - 1) / kGroups;
  for (uint64_t block = blockIdx.x; block < a.blocks; block += gridDim.x) {
    if (block < sums) {
      const uint64_t unit = block * kGroups + group;
      if (unit >= a.units) continue;
      const uint32_t t = (uint32_t)(unit / a.strips), strip = (uint32_t)(unit - t * a.strips), lane = threadIdx.x % kLanes;
      const uint32_t c = (strip * kLanes + lane) * CH;
      Tile<W, R, kDivide, kAdd, CH, kLanes>{a, c, lane, (int)(a.cols - c)}.run(t);
    } else {
      const uint32_t lane = threadIdx.x % a.clear_lanes;
      const uint64_t id = (block - sums) * (256 / a.clear_lanes) + threadIdx.x / a.clear_lanes;
      if (id < a.vocab && (!a.first || a.first[id] == a.first[id + 1]))
        clear_row((char *)((W *)a.dtable + id * a.lddt), (uint64_t)a.cols * sizeof(W), sizeof(W), lane, a.clear_lanes);
    }
  }
}

// The tokens that go past the end of the tile where they begin, blockIdx.y: their lines, in order.  A thread
// adds all of a token's lines at its column, eight loads ahead: 6 us where text-like tokens have 16384 rows of
// 4096 bf16 columns, but about 50 ns a line where one token has very many (f32, 64 columns, tiles of 8: 26 us
// for its 4096 rows, 418 for 65536).
template <class W, bool kAdd>
__global__ __launch_bounds__(256) void k_join(GradArgs a) {
  const uint64_t pitch = line_pitch(a.cols);
  const uint32_t all = a.first[a.vocab], lane = threadIdx.x & 63;
  for (uint32_t t = blockIdx.y; t < a.tiles; t += gridDim.y) {
    const uint32_t t0 = t * a.tile, t1 = t0 + a.tile;
    if (t1 >= all) return;
    const uint64_t begins = __ballot(lane < a.tile && a.run[t0 + (lane < a.tile ? lane : 0)] != 0);
    if (!begins) continue;
    const uint32_t begin = t0 + 63 - (uint32_t)__clzll((long long)begins), end = begin + a.run[begin];
    if (end <= t1) continue;
    const uint32_t last = (end - 1) / a.tile;
    W *out = (W *)a.dtable + (uint32_t)token(a.ids, a.ids64, a.order[begin]) * a.lddt;
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
      sum *= a.scale;
      out[c] = (W)(kAdd ? sum + (float)out[c] : sum);
    }
  }
}

// ---------------------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------------------
// Places to a tile: 8, 16, 32 or 64, the most that leave kUnits waves' work, eight to a compute unit (and no
// more than the lanes of a strip, which hold them).  More units leave more partial lines, fewer leave compute
// units without work.  The gradient's us, bf16, rows evenly spread and text-like, with 1024, 2048 and 4096 units:
//     65536x256  of 32768 tokens  48.4 45.8 50.2    74.3 77.1 90.7
//     16384x1024                  31.5 34.6 37.8    35.9 38.8 43.7
//     65536x1024                  80.4 80.0 85.9     101  101  105
//     16384x4096                  98.3 98.2  101    93.4 93.9 95.8
//     4096x1024, 65536x4096, 2047x1001 of 50001: within 1 %
constexpr uint64_t kUnits = 2048;

struct TilePlan {
  uint64_t tile = 8, strips, least;  // least: tiles that make kUnits
  uint32_t lanes;
  TilePlan(uint64_t rows, uint64_t cols, uint64_t chunk) {
    const uint64_t ch = cols < chunk ? 1 : chunk;
    lanes = cols <= 8 * ch ? 8 : cols <= 16 * ch ? 16 : cols <= 32 * ch ? 32 : 64;
    strips = (cols + lanes * ch - 1) / (lanes * ch);
    least = (kUnits * 64 / lanes + strips - 1) / strips;
    while (tile < lanes && rows >= 2 * tile * least) tile *= 2;
  }
  uint64_t tiles(uint64_t rows) const { return (rows + tile - 1) / tile; }
  // The most tiles that any number of rows up to this one makes: below 2 * least where a wider tile follows.
  uint64_t room(uint64_t rows) const {
    const uint64_t n = tiles(rows);
    return tile > 8 && n < 2 * least ? 2 * least : n;
  }
};

static uint64_t embedding_bytes(uint64_t rows, uint64_t cols, uint64_t vocab) {
  if (rows == 0 || cols == 0 || vocab == 0) return 0;
  uint64_t room = 0;
  for (uint64_t chunk = 4; chunk <= 8; chunk += 4) {  // one size serves every type
    const uint64_t n = TilePlan(rows, cols, chunk).room(rows);
    room = n > room ? n : room;
  }
  return 4 * (2 * rows + vocab + 1) + 8 * room * line_pitch(cols) + 12;  // 12: the lines are aligned to 16 bytes
}

constexpr int kLookupChunks = 2;

template <class W, class R, bool kDivide>
struct Embedding {
  static constexpr int CH = kChunk<W, R>;

  static tk_status forward(LookupArgs a, uint64_t rows, hipStream_t s) {
    constexpr int V = kLookupChunks;
    const int ch = a.cols < (uint32_t)CH ? 1 : CH;
    const bool wide = a.cols >= 64u * CH;
    a.chunks_per_row = (a.cols + ch - 1) / ch;
    if (wide) a.chunks_per_row = (a.chunks_per_row + 64 * V - 1) / (64 * V);
    a.per_row = Divisor(a.chunks_per_row);
    const uint64_t rows_each = (wide ? 1ull << 25 : 1ull << 30) / a.chunks_per_row;
    for (uint64_t r = 0; r < rows; r += rows_each) {
      a.row0 = r;
      a.chunks = (uint32_t)((rows - r < rows_each ? rows - r : rows_each) * a.chunks_per_row);
      const auto go = [&](auto kernel, uint32_t each) {
        hipLaunchKernelGGL(kernel, dim3((a.chunks + each - 1) / each), dim3(256), 0, s, a);
      };
      if (ch == 1) go(k_embedding<W, R, kDivide, 1, false, 1>, 256);
      else if (wide) go(k_embedding<W, R, kDivide, CH, true, V>, 4);
      else go(k_embedding<W, R, kDivide, CH, false, 1>, 256);
      const tk_status st = launch_status();
      if (st != TK_OK) return st;
    }
    return TK_OK;
  }

  template <bool kAdd, int ch, int kLanes>
  static void launch_sums(GradArgs a, hipStream_t s) {
    constexpr uint32_t kGroups = 256 / kLanes;
    a.blocks = (a.units + kGroups - 1) / kGroups;
    if (!kAdd) {
      // Two vectors to a lane, where a row is that long.  Runs of absent rows cleared as one by a work-group,
      // 8, 16 or 32 KiB to each, take 93.2, 98.1 and 103.6 us for 92.9 (16384 tokens of 32768, 4096 columns, bf16).
      const uint64_t vectors = (uint64_t)a.cols * sizeof(W) / 16;
      a.clear_lanes = 8;
      while (a.clear_lanes < 256 && a.clear_lanes * 2 < vectors) a.clear_lanes *= 2;
      a.blocks += ((uint64_t)a.vocab + 256 / a.clear_lanes - 1) / (256 / a.clear_lanes);
    }
    const uint64_t most = 1ull << 23;  // a launch holds fewer than 2^32 threads
    hipLaunchKernelGGL((k_token_sums<W, R, kDivide, kAdd, ch, kLanes>), dim3((uint32_t)(a.blocks < most ? a.blocks : most)),
                       dim3(256), 0, s, a);
  }
  template <bool kAdd>
  static tk_status sums(GradArgs a, hipStream_t s) {
    const TilePlan p(a.rows, a.cols, CH);
    a.tile = (uint32_t)p.tile;
    a.tiles = (uint32_t)p.tiles(a.rows);
    a.strips = p.strips;
    a.units = a.tiles * p.strips;
    if (a.cols < (uint32_t)CH) launch_sums<kAdd, 1, 8>(a, s);
    else if (p.lanes == 8) launch_sums<kAdd, CH, 8>(a, s);
    else if (p.lanes == 16) launch_sums<kAdd, CH, 16>(a, s);
    else if (p.lanes == 32) launch_sums<kAdd, CH, 32>(a, s);
    else launch_sums<kAdd, CH, 64>(a, s);
    const tk_status st = launch_status();
    if (st != TK_OK || a.tiles <= 1) return st;
    const uint32_t blocks = (a.cols + 255) / 256;
    hipLaunchKernelGGL((k_join<W, kAdd>), dim3(blocks < 1024 ? blocks : 1024, a.tiles < 8192 ? a.tiles : 8192), dim3(256), 0, s, a);
    return launch_status();
  }
  static tk_status backward(const GradArgs &a, bool add, hipStream_t s) { return add ? sums<true>(a, s) : sums<false>(a, s); }
};

static tk_status sort_tokens(SortArgs a, hipStream_t s) {
  const auto go = [&](auto kernel, uint32_t range) {
    a.ranges = (a.vocab + range - 1) / range;
    hipLaunchKernelGGL(kernel, dim3(a.ranges < 1u << 16 ? a.ranges : 1u << 16), dim3(64 * kSortWaves), 0, s, a);
  };
  // The smallest range that makes one work-group to a compute unit, as each reads all rows: the fewer
  // tokens it has, the fewer of the rows are its own (23233 rows of 1533 tokens, text-like, with a range
  // of 8 and of 64: 16.1 and 19.4 us).
  const bool wide = a.ids64;
  if (a.vocab <= 8 * 256) go(wide ? k_sort_tokens<8, true> : k_sort_tokens<8, false>, 8);
  else if (a.vocab <= 32 * 256) go(wide ? k_sort_tokens<32, true> : k_sort_tokens<32, false>, 32);
  else if (a.vocab <= 128 * 256) go(wide ? k_sort_tokens<128, true> : k_sort_tokens<128, false>, 128);
  else go(wide ? k_sort_tokens<512, true> : k_sort_tokens<512, false>, 512);
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
    uint32_t *order = (uint32_t *)workspace, *run = order + rows, *first = run + rows;
    a.order = order; a.run = run; a.first = first;
    a.partial = (float *)(((uintptr_t)(first + vocab + 1) + 15) & ~(uintptr_t)15);
    if ((st = sort_tokens(SortArgs{ids, order, run, first, a.rows, a.vocab, 0, a.ids64}, stream)) != TK_OK) return st;
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
