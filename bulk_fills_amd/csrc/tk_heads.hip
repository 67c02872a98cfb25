// tk_heads.hip -- the norm of each query and key head with the position rotation in the same pass,
// and its gradient.
#include <type_traits>

#include "tk_row_checks.h"
#include "tk_rows.h"

namespace tk {

// A side is the queries or the keys: `heads` heads of `dim` elements, one after the other in a row.
struct Side {
  const void *x, *dy, *gamma;
  void *out;  // y, or dx
  uint64_t ldx, lddy, ldo;
  uint32_t heads, units;  // units of work of a row
  Divisor by_units;
};

struct HeadArgs {
  Side side[2];
  const void *positions;
  const float *cosines, *sines;
  float *partial;  // lines of partial sums: dgamma_q's, then dgamma_k's
  uint64_t rows, table_rows;
  uint32_t dim, half, pair_slots, slots;
  uint32_t waves_q;  // of a backward work-group's waves those for the queries
  float eps;
  bool i64, params_f32, once;  // once: the call's reads go past the caches
};

// ---- a lane's part of a head ----
// A lane holds a slot, twice P elements of its head.  The first slots hold pairs: with halves paired,
// P elements of the first half and their partners, and with neighbours paired 2 P in a row.  The rest
// of the head, which does not turn, follows in slots of 2 P in a row.  So a pair never leaves its
// lane, and with a head's width a multiple of 4 P every access is a whole vector.
struct Slot {
  uint32_t at1, at2, angle;  // first elements of its two vectors, and the first pair's angle
  int n1, n2, pairs;         // how many elements count; pairs: 0 in the slots that do not turn
};

template <int P, bool kNeighbours>
__device__ __forceinline__ Slot slot_of(const HeadArgs &a, uint32_t s) {
  const auto upto = [](int n) { return n < 0 ? 0 : n < P ? n : P; };
  Slot t{};
  if (s >= a.slots) return t;
  if (s >= a.pair_slots) {
    t.at1 = 2 * a.half + (s - a.pair_slots) * 2 * P;
    t.at2 = t.at1 + P;
    t.n1 = upto((int)a.dim - (int)t.at1);
    t.n2 = upto((int)a.dim - (int)t.at2);
    return t;
  }
  t.angle = s * P;
  t.pairs = upto((int)a.half - (int)t.angle);
  if (kNeighbours) {
    t.at1 = 2 * t.angle;
    t.at2 = t.at1 + P;
    t.n1 = upto(2 * t.pairs);
    t.n2 = 2 * t.pairs - t.n1;
  } else {
    t.at1 = t.angle;
    t.at2 = a.half + t.angle;
    t.n1 = t.n2 = t.pairs;
  }
  return t;
}

// n of P elements as floats, the others 0.  Fewer than P are loaded one by one: a vector would reach
// into what the call need not own.
template <int P, class T>
__device__ __forceinline__ void load_some(const T *p, int n, float *v) {
  if (n == P) {
    const Chunk<T, P> t = *(const Chunk<T, P> *)p;
#pragma unroll
    for (int e = 0; e < P; ++e) v[e] = (float)t[e];
  } else {
#pragma unroll
    for (int e = 0; e < P; ++e) v[e] = e < n ? (float)p[e] : 0.0f;
  }
}

// Both vectors of a slot, at a head's first element.
template <int P, class T>
__device__ __forceinline__ void load_slot(const void *head, const Slot &s, float *v) {
  load_some<P, T>((const T *)head + s.at1, s.n1, v);
  load_some<P, T>((const T *)head + s.at2, s.n2, v + P);
}

template <int P, class T>
__device__ __forceinline__ void store_slot(void *head, const Slot &s, const float *v) {
  store_chunk<P>((T *)head + s.at1, s.n1, v);
  store_chunk<P>((T *)head + s.at2, s.n2, v + P);
}

template <int P, class T>
__device__ __forceinline__ void load_gamma(const HeadArgs &a, const void *gamma, const Slot &s, float *v) {
  if (!gamma) {
#pragma unroll
    for (int e = 0; e < 2 * P; ++e) v[e] = 1.0f;
  } else if (a.params_f32) {
    load_slot<P, float>(gamma, s, v);
  } else {
    load_slot<P, T>(gamma, s, v);
  }
}

// The position of a row; beyond any table where it is negative.
__device__ __forceinline__ uint64_t position(const HeadArgs &a, uint64_t row) {
  if (!a.positions) return row;
  return a.i64 ? (uint64_t)((const int64_t *)a.positions)[row] : (uint64_t)(int64_t)((const int32_t *)a.positions)[row];
}

// The angles of a position for a slot.  A row whose position is none of the tables' does not turn.
template <int P>
struct Angles {
  float c[P], s[P];
  bool turns;
  __device__ __forceinline__ void load(const HeadArgs &a, uint64_t at, const Slot &t) {
    turns = t.pairs > 0 && at < a.table_rows;
    const uint64_t from = turns ? at * a.half + t.angle : 0;
    const int n = turns ? t.pairs : 0;
    load_some<P, float>(a.cosines + from, n, c);
    load_some<P, float>(a.sines + from, n, s);
  }
  // v's pairs turned by the angles, or back.
  template <bool kNeighbours, bool kBack>
  __device__ __forceinline__ void turn(float *v) const {
    if (!turns) return;
#pragma unroll
    for (int e = 0; e < P; ++e) {
      float &x = kNeighbours ? v[2 * e] : v[e], &y = kNeighbours ? v[2 * e + 1] : v[P + e];
      const float sine = kBack ? -s[e] : s[e], u = x;
      x = __builtin_fmaf(-y, sine, u * c[e]);
      y = __builtin_fmaf(u, sine, y * c[e]);
    }
  }
};

// A slot's two vectors as loaded, and their elements as floats.  Fewer than P are loaded one by one.
template <bool kOnce, int P, class T>
struct Raw {
  Chunk<T, P> v[2];
  __device__ __forceinline__ void load(const void *head, const Slot &s) {
    load_one((const T *)head + s.at1, s.n1, v[0]);
    load_one((const T *)head + s.at2, s.n2, v[1]);
  }
  __device__ __forceinline__ void floats(float *x) const {
#pragma unroll
    for (int e = 0; e < P; ++e) {
      x[e] = (float)v[0][e];
      x[P + e] = (float)v[1][e];
    }
  }

 private:
  static __device__ __forceinline__ void load_one(const T *p, int n, Chunk<T, P> &t) {
    if (n == P) {
      t = load_chunk<kOnce, P>(p);
    } else {
#pragma unroll
      for (int e = 0; e < P; ++e) t[e] = e < n ? p[e] : (T)0.0f;
    }
  }
};

// ---- kernels ----
// A wave takes up to S steps of one row's queries or keys, a step being 64 / kLanes heads of kLanes lanes
// each: all of its loads are on their way before the first value is used, and the angles and gamma serve
// all steps.  blockIdx.y counts the queries' steps of a row by S, then the keys' (a row's units beside each
// other take 73 us for 64).
//
// Bound by memory: bf16 16384x(32+8)x128 from a projection's rows 63.6 us, 5.3 TB/s (through the caches 68, with
// two steps 69, with heads one after the other 79).
template <class T, int P, int kLanes, bool kNeighbours, bool kOnce, int S>
__global__ __launch_bounds__(256) void k_heads(HeadArgs a) {
  constexpr uint32_t kGroups = 64 / kLanes;
  const uint32_t group = (threadIdx.x & 63) / kLanes;
  const Slot slot = slot_of<P, kNeighbours>(a, threadIdx.x % kLanes);
  const float inv = 1.0f / (float)a.dim;
  const uint64_t first = blockIdx.x * 4ull + (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  for (uint32_t unit = blockIdx.y; unit < a.side[0].units + a.side[1].units; unit += gridDim.y) {
    const bool key = unit >= a.side[0].units;
    const Side &side = a.side[key];
    const uint32_t h0 = (key ? unit - a.side[0].units : unit) * (S * kGroups) + group;
    float g[2 * P];
    load_gamma<P, T>(a, side.gamma, slot, g);
    for (uint64_t row = first; row < a.rows; row += gridDim.x * 4ull) {
      Raw<kOnce, P, T> x[S];
      Angles<P> angles;
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (h0 + s * kGroups < side.heads) x[s].load((const T *)side.x + row * side.ldx + (h0 + s * kGroups) * a.dim, slot);
      angles.load(a, position(a, row), slot);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if (h0 + s * kGroups >= side.heads) break;
        float v[2 * P], sum = 0.0f;
        x[s].floats(v);
#pragma unroll
        for (int e = 0; e < 2 * P; ++e) sum = __builtin_fmaf(v[e], v[e], sum);
        const float rstd = rsqrt_any(__builtin_fmaf(lanes_sum<kLanes>(sum), inv, a.eps));
#pragma unroll
        for (int e = 0; e < 2 * P; ++e) v[e] = v[e] * rstd * g[e];
        angles.template turn<kNeighbours, false>(v);
        store_slot<P, T>((T *)side.out + row * side.ldo + (h0 + s * kGroups) * a.dim, slot, v);
      }
    }
  }
}

// The sum over a wave's lanes that hold the same slot, in all of them.
template <int kLanes>
__device__ __forceinline__ float slots_sum(float x) {
  if (kLanes <= 1) x += dpp<0x121>(x);  // row_ror:1, 2, 4, 8
  if (kLanes <= 2) x += dpp<0x122>(x);
  if (kLanes <= 4) x += dpp<0x124>(x);
  if (kLanes <= 8) x += dpp<0x128>(x);
  if (kLanes <= 16) x = swap_sum16(x);
  if (kLanes <= 32) x = swap_sum32(x);
  return x;
}

constexpr int kBackWaves = 16, kFlight = 2;

// The gradient: one pass over x and dy, the statistics made anew.  The waves of a work-group are shared
// out between queries and keys, a.waves_q for those, so that each keeps one gamma and its gradient's sums
// in registers over all its rows; at the end a work-group's sums go to the workspace as one line for each.
// A wave goes from step to step through all rows.  Bound by the time that its loads take: two steps are on
// their way, and the next one's position (bf16 8192x(32+8)x128 53.8 us; one step, and all of a row's to
// a wave, 64; three and four steps 55.6).  Four elements to a vector rather than eight leave the
// registers for that.
template <class T, int P, int kLanes, bool kNeighbours, bool kOnce>
__global__ __launch_bounds__(64 * kBackWaves) void k_heads_bwd(HeadArgs a) {
  constexpr uint32_t kGroups = 64 / kLanes;
  constexpr int kAhead = P > 4 ? 1 : kFlight;
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), group = (threadIdx.x & 63) / kLanes;
  const Slot slot = slot_of<P, kNeighbours>(a, threadIdx.x % kLanes);
  const float inv = 1.0f / (float)a.dim;
  const bool key = wave >= a.waves_q;
  const Side &side = a.side[key];
  const uint32_t waves = key ? kBackWaves - a.waves_q : a.waves_q, stride = gridDim.x * waves;
  const uint32_t units = (uint32_t)a.rows * side.units;  // steps of all rows
  float acc[2 * P], g[2 * P];
#pragma unroll
  for (int e = 0; e < 2 * P; ++e) acc[e] = 0.0f;
  load_gamma<P, T>(a, side.gamma, slot, g);
  Raw<kOnce, P, T> in_x[kAhead], in_d[kAhead];
  Angles<P> angles[kAhead];
  uint32_t unit = blockIdx.x * waves + (key ? wave - a.waves_q : wave), loaded = unit;
  uint64_t pos = loaded < units ? position(a, side.by_units.of(loaded)) : 0;
  // The head of this lane's group in a step: the row, and the head's first element.  Groups behind the
  // last head load it too.
  const auto load = [&](int k) {
    if (loaded < units) {
      const uint32_t row = side.by_units.of(loaded), h = (loaded - row * side.units) * kGroups + group;
      const uint32_t at = (h < side.heads ? h : side.heads - 1) * a.dim;
      in_x[k].load((const T *)side.x + row * side.ldx + at, slot);
      in_d[k].load((const T *)side.dy + row * side.lddy + at, slot);
      angles[k].load(a, pos, slot);
    }
    loaded += stride;
    if (loaded < units) pos = position(a, side.by_units.of(loaded));
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) load(k);
  while (unit < units) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (unit >= units) break;
      const uint32_t row = side.by_units.of(unit), h = (unit - row * side.units) * kGroups + group;
      float x[2 * P], d[2 * P], s[2] = {0.0f, 0.0f};
      in_x[k].floats(x);
      in_d[k].floats(d);
      angles[k].template turn<kNeighbours, true>(d);
      load(k);
      unit += stride;
      const bool here = h < side.heads;
#pragma unroll
      for (int e = 0; e < 2 * P; ++e) s[0] = __builtin_fmaf(x[e], x[e], s[0]);
      const float rstd = rsqrt_any(__builtin_fmaf(lanes_sum<kLanes>(s[0]), inv, a.eps));
#pragma unroll
      for (int e = 0; e < 2 * P; ++e) {
        x[e] *= rstd;  // h
        const float to = __builtin_fmaf(d[e], x[e], acc[e]);
        acc[e] = here ? to : acc[e];
        d[e] *= g[e];
        s[1] = __builtin_fmaf(d[e], x[e], s[1]);
      }
      const float m = lanes_sum<kLanes>(s[1]) * inv;
#pragma unroll
      for (int e = 0; e < 2 * P; ++e) d[e] = rstd * __builtin_fmaf(-x[e], m, d[e]);
      if (here) store_slot<P, T>((T *)side.out + row * side.ldo + h * a.dim, slot, d);
    }
  }
  if (!a.partial) return;
  __shared__ float tile[kBackWaves][kLanes * 2 * P];
#pragma unroll
  for (int e = 0; e < 2 * P; ++e) {
    const float v = slots_sum<kLanes>(acc[e]);
    if ((threadIdx.x & 63) < kLanes) tile[wave][(threadIdx.x & 63) * 2 * P + e] = v;
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < 2 * kLanes * 2 * P; i += 64 * kBackWaves) {
    const uint32_t k = i / (kLanes * 2 * P), n = i % (kLanes * 2 * P), from = k ? a.waves_q : 0, to = k ? kBackWaves : a.waves_q;
    const Slot t = slot_of<P, kNeighbours>(a, n / (2 * P));
    const int e = (int)(n % (2 * P));
    float v = 0.0f;
    for (uint32_t w = from; w < to; ++w) v += tile[w][n];
    float *line = a.partial + ((uint64_t)k * gridDim.x + blockIdx.x) * line_pitch(a.dim);
    if (e < P) {
      if (e < t.n1) line[t.at1 + e] = v;
    } else if (e - P < t.n2) {
      line[t.at2 + e - P] = v;
    }
  }
}

// ---- launches ----
constexpr int kSteps = 4, kForwardP = 8;
constexpr uint64_t kMostDim = 512;  // 64 lanes of 8 f32 elements

template <class T>
struct Heads {
  template <int P, int kLanes, bool kNeighbours, bool kOnce, int S>
  static void forward(HeadArgs a, hipStream_t s) {
    for (Side &side : a.side) side.units = (side.heads + S * (64 / kLanes) - 1) / (S * (64 / kLanes));
    const uint64_t x = (a.rows + 3) / 4, y = (uint64_t)a.side[0].units + a.side[1].units;
    hipLaunchKernelGGL((k_heads<T, P, kLanes, kNeighbours, kOnce, S>),
                       dim3((uint32_t)(x < 1u << 20 ? x : 1u << 20), (uint32_t)(y < 4096 ? y : 4096)), dim3(256), 0, s, a);
  }
  template <int P, int kLanes, bool kNeighbours>
  static uint32_t backward(HeadArgs a, hipStream_t s) {
    constexpr uint32_t kGroups = 64 / kLanes;
    const uint64_t steps[2] = {(a.side[0].heads + kGroups - 1) / kGroups, (a.side[1].heads + kGroups - 1) / kGroups};
    // the waves by the steps, at least one for a side that has any
    const uint64_t both = steps[0] + steps[1];
    uint64_t q = (kBackWaves * steps[0] + both / 2) / both;
    if (q == 0 && steps[0]) q = 1;
    if (q == kBackWaves && steps[1]) --q;
    a.waves_q = (uint32_t)q;
    uint64_t grid = 1;
    for (int k = 0; k < 2; ++k) {
      if (!steps[k]) continue;
      const uint64_t waves = k ? kBackWaves - q : q;
      a.side[k].units = (uint32_t)steps[k];
      a.side[k].by_units = Divisor(steps[k]);
      const uint64_t sets = (a.rows * steps[k] + waves - 1) / waves;
      grid = sets > grid ? sets : grid;
    }
    if (grid > kMaxLines) grid = kMaxLines;
    const dim3 g((uint32_t)grid), b(64 * kBackWaves);
    if (a.once) hipLaunchKernelGGL((k_heads_bwd<T, P, kLanes, kNeighbours, true>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_heads_bwd<T, P, kLanes, kNeighbours, false>), g, b, 0, s, a);
    return (uint32_t)grid;
  }
  // Four steps to a wave where that leaves enough waves.  us, with four and with one: bf16 (32+8)x128, of 5
  // steps, 8 rows 5.2 4.4, 512 5.5 4.9, 1024 6.6 6.8, 2048 9.7 11.5, 4096 16.7 19.2.  Few heads have no four steps
  // to a side: 8192x(8+2)x64 bf16 15.2 13.7, f32 13.1 12.1, which the rule leaves.
  template <int P, int kLanes, bool kNeighbours>
  static void forward_by(const HeadArgs &a, hipStream_t s) {
    constexpr uint64_t kGroups = 64 / kLanes;
    const uint64_t steps = (a.side[0].heads + kGroups - 1) / kGroups + (a.side[1].heads + kGroups - 1) / kGroups;
    if (a.once) forward<P, kLanes, kNeighbours, true, kSteps>(a, s);
    else if (a.rows * steps >= 8192) forward<P, kLanes, kNeighbours, false, kSteps>(a, s);
    else forward<P, kLanes, kNeighbours, false, 1>(a, s);
  }
  static void set_slots(HeadArgs &a, uint32_t P) {
    a.pair_slots = (a.half + P - 1) / P;
    a.slots = a.pair_slots + (a.dim - 2 * a.half + 2 * P - 1) / (2 * P);
  }
  // The work-groups that ran (backward), with the lanes that a head's slots need.
  template <int P, bool kNeighbours, bool kBack, int kLanes = 2>
  static uint32_t lanes(const HeadArgs &a, hipStream_t s) {
    if constexpr (kLanes < 64)
      if (a.slots > kLanes) return lanes<P, kNeighbours, kBack, 2 * kLanes>(a, s);
    if constexpr (kBack) return backward<P, kLanes, kNeighbours>(a, s);
    else forward_by<P, kLanes, kNeighbours>(a, s);
    return 0;
  }
  template <bool kNeighbours, bool kBack>
  static uint32_t run(HeadArgs a, hipStream_t s) {
    constexpr int P = kBack || sizeof(T) == 4 ? 4 : kForwardP;
    set_slots(a, P);
    if (P < 8 && a.slots > 64) {  // the widest heads, of which some elements turn and some do not
      set_slots(a, 8);
      return lanes<8, kNeighbours, kBack, 64>(a, s);
    }
    return lanes<P, kNeighbours, kBack>(a, s);
  }
};

constexpr uint32_t kHeadFlags = TK_PARAMS_F32 | TK_INDEX_I64 | TK_INTERLEAVED;
constexpr int kQueries = 1, kKeys = 2;  // Region's kinds

struct HeadCall {
  RowType type;
  uint64_t rows, heads_q, heads_k, dim, rotary;
  float eps;
  uint32_t flags;
  HeadArgs a{};

  uint64_t width(int k) const { return (k ? heads_k : heads_q) * dim; }
  tk_status check_numbers() const {
    if (!(eps >= 0.0f && eps < INFINITY) || (flags & ~kHeadFlags) || rotary % 2 || rotary > dim) return TK_EINVAL;
    if (rows >= kMaxDim || dim > kMostDim || heads_q >= kMaxDim || heads_k >= kMaxDim) return TK_ERANGE;
    if ((heads_q + heads_k) * dim >= kMaxDim || rows * (heads_q + heads_k) >= kMaxDim) return TK_ERANGE;
    return TK_OK;
  }
  bool empty() const { return rows == 0 || dim == 0 || heads_q + heads_k == 0; }
  // The arguments that both directions have.
  tk_status angles(Arguments &c, const void *positions, uint64_t table_rows, const float *cosines, const float *sines) {
    if (table_rows >= kMaxDim) return TK_ERANGE;
    c.vector(positions, rows, flags & TK_INDEX_I64 ? 8 : 4, false, false);
    if (rotary && table_rows) {
      c.vector(cosines, table_rows * (rotary / 2), 4, false, true);
      c.vector(sines, table_rows * (rotary / 2), 4, false, true);
    }
    a.positions = positions; a.table_rows = table_rows; a.cosines = cosines; a.sines = sines;
    a.rows = rows; a.side[0].heads = (uint32_t)heads_q; a.side[1].heads = (uint32_t)heads_k;
    a.dim = (uint32_t)dim; a.half = (uint32_t)(rotary / 2); a.eps = eps;
    a.i64 = flags & TK_INDEX_I64; a.params_f32 = params_f32(type, flags);
    return TK_OK;
  }
  uint32_t run(bool back, hipStream_t s) const {
    const auto by_type = [&](auto h) {
      typedef Heads<decltype(h)> K;
      if (flags & TK_INTERLEAVED) return back ? K::template run<true, true>(a, s) : K::template run<true, false>(a, s);
      return back ? K::template run<false, true>(a, s) : K::template run<false, false>(a, s);
    };
    return type == kF32 ? by_type(float()) : type == kF16 ? by_type(f16_t()) : by_type(bf16_t());
  }
};

static tk_status head_forward(HeadCall h, const void *q, uint64_t ldq, const void *k, uint64_t ldk, const void *gamma_q,
                              const void *gamma_k, const void *positions, uint64_t table_rows, const float *cosines,
                              const float *sines, void *yq, uint64_t ldyq, void *yk, uint64_t ldyk, hipStream_t stream) {
  tk_status st = h.check_numbers();
  if (st != TK_OK || h.empty()) return st;
  Arguments c{h.type, h.rows, h.dim, h.flags};
  const void *x[2] = {q, k}, *gamma[2] = {gamma_q, gamma_k};
  void *y[2] = {yq, yk};
  const uint64_t ldx[2] = {ldq, ldk}, ldy[2] = {ldyq, ldyk};
  for (int i = 0; i < 2; ++i) {
    if (!h.width(i)) continue;
    c.matrix_of(x[i], h.rows, h.width(i), ldx[i], c.t(), false, true, i ? kKeys : kQueries);
    c.matrix_of(y[i], h.rows, h.width(i), ldy[i], c.t(), true, true, i ? kKeys : kQueries);
    c.vector(gamma[i], h.dim, c.par(), false, false);
    h.a.side[i] = Side{x[i], nullptr, gamma[i], y[i], ldx[i], 0, ldy[i], 0, 0, {}};
  }
  if ((st = h.angles(c, positions, table_rows, cosines, sines)) != TK_OK || (st = c.done()) != TK_OK) return st;
  h.a.once = h.rows * (h.width(0) + h.width(1)) * c.t() > kCachedReads;
  h.run(false, stream);
  return launch_status();
}

static uint64_t head_bytes(uint64_t rows, uint64_t heads_q, uint64_t heads_k, uint64_t dim) {
  return rows * (heads_q + heads_k) * dim ? 8 * kMaxLines * line_pitch(dim) : 0;
}

static tk_status head_backward(HeadCall h, const void *dyq, uint64_t lddyq, const void *dyk, uint64_t lddyk, const void *q,
                               uint64_t ldq, const void *k, uint64_t ldk, const void *gamma_q, const void *gamma_k,
                               const void *positions, uint64_t table_rows, const float *cosines, const float *sines,
                               void *dq, uint64_t lddq, void *dk, uint64_t lddk, void *dgamma_q, void *dgamma_k,
                               void *workspace, uint64_t bytes, hipStream_t stream) {
  tk_status st = h.check_numbers();
  if (st != TK_OK || h.dim == 0) return st;
  Arguments c{h.type, h.rows, h.dim, h.flags};
  const bool sums = dgamma_q || dgamma_k;
  c.vector(dgamma_q, h.dim, c.par(), true, false);
  c.vector(dgamma_k, h.dim, c.par(), true, false);
  if (h.empty()) {
    if ((st = c.done()) != TK_OK || !sums) return st;
    return finish(h.type, h.flags, nullptr, 0, h.dim, dgamma_q, dgamma_k, nullptr, stream);
  }
  const void *x[2] = {q, k}, *dy[2] = {dyq, dyk}, *gamma[2] = {gamma_q, gamma_k};
  void *dx[2] = {dq, dk};
  const uint64_t ldx[2] = {ldq, ldk}, lddy[2] = {lddyq, lddyk}, lddx[2] = {lddq, lddk};
  for (int i = 0; i < 2; ++i) {
    if (!h.width(i)) continue;
    const int kind = i ? kKeys : kQueries;
    c.matrix_of(x[i], h.rows, h.width(i), ldx[i], c.t(), false, true, kind);
    c.matrix_of(dy[i], h.rows, h.width(i), lddy[i], c.t(), false, true, kind);
    c.matrix_of(dx[i], h.rows, h.width(i), lddx[i], c.t(), true, true, kind);
    c.vector(gamma[i], h.dim, c.par(), false, false);
    h.a.side[i] = Side{x[i], dy[i], gamma[i], dx[i], ldx[i], lddy[i], lddx[i], 0, 0, {}};
  }
  const uint64_t need = sums ? head_bytes(h.rows, h.heads_q, h.heads_k, h.dim) : 0;
  if (!serves(workspace, bytes, need)) return TK_EINVAL;
  if (need) c.vector(workspace, need / 4, 4, true, true);
  if ((st = h.angles(c, positions, table_rows, cosines, sines)) != TK_OK || (st = c.done()) != TK_OK) return st;
  h.a.partial = sums ? (float *)workspace : nullptr;
  h.a.once = h.rows * (h.width(0) + h.width(1)) * 2 * c.t() > kCachedReads;
  const uint32_t lines = h.run(true, stream);
  if ((st = launch_status()) != TK_OK || !sums) return st;
  return finish(h.type, h.flags, h.a.partial, lines, h.dim, dgamma_q, dgamma_k, nullptr, stream);
}

}  // namespace tk

extern "C" {

tk_status tk_head_norm_workspace_bytes(uint64_t rows, uint64_t heads_q, uint64_t heads_k, uint64_t dim, uint64_t *bytes) {
  if (!bytes) return TK_EINVAL;
  if (rows >= tk::kMaxDim || heads_q >= tk::kMaxDim || heads_k >= tk::kMaxDim || dim > tk::kMostDim ||
      (heads_q + heads_k) * dim >= tk::kMaxDim || rows * (heads_q + heads_k) >= tk::kMaxDim)
    return TK_ERANGE;
  *bytes = tk::head_bytes(rows, heads_q, heads_k, dim);
  return TK_OK;
}

#define TK_HEADS(SUFFIX, TYPE)                                                                                            \
  tk_status tk_head_norm_rotate_##SUFFIX(                                                                                 \
      uint64_t rows, uint64_t heads_q, uint64_t heads_k, uint64_t dim, uint64_t rotary, float eps, uint32_t flags,        \
      const void *q, uint64_t ldq, const void *k, uint64_t ldk, const void *gamma_q, const void *gamma_k,                 \
      const void *positions, uint64_t table_rows, const float *cosines, const float *sines, void *yq, uint64_t ldyq,      \
      void *yk, uint64_t ldyk, hipStream_t stream) {                                                                      \
    return tk::head_forward(tk::HeadCall{TYPE, rows, heads_q, heads_k, dim, rotary, eps, flags}, q, ldq, k, ldk, gamma_q, \
                            gamma_k, positions, table_rows, cosines, sines, yq, ldyq, yk, ldyk, stream);                  \
  }                                                                                                                       \
  tk_status tk_head_norm_rotate_backward_##SUFFIX(                                                                        \
      uint64_t rows, uint64_t heads_q, uint64_t heads_k, uint64_t dim, uint64_t rotary, float eps, uint32_t flags,        \
      const void *dyq, uint64_t lddyq, const void *dyk, uint64_t lddyk, const void *q, uint64_t ldq, const void *k,       \
      uint64_t ldk, const void *gamma_q, const void *gamma_k, const void *positions, uint64_t table_rows,                 \
      const float *cosines, const float *sines, void *dq, uint64_t lddq, void *dk, uint64_t lddk, void *dgamma_q,         \
      void *dgamma_k, void *workspace, uint64_t workspace_bytes, hipStream_t stream) {                                    \
    return tk::head_backward(tk::HeadCall{TYPE, rows, heads_q, heads_k, dim, rotary, eps, flags}, dyq, lddyq, dyk, lddyk, \
                             q, ldq, k, ldk, gamma_q, gamma_k, positions, table_rows, cosines, sines, dq, lddq, dk, lddk, \
                             dgamma_q, dgamma_k, workspace, workspace_bytes, stream);                                     \
  }

TK_HEADS(f32, tk::kF32)
TK_HEADS(f16, tk::kF16)
TK_HEADS(bf16, tk::kBF16)

}  // extern "C"
