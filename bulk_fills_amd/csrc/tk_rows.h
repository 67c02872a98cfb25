// tk_rows.h -- kernels of the row operators (dropout-add, layer norm, both fused) for one
// pair of types: T of the activations, R of the residual stream.  Instantiated by
// tk_rows_{f32,f16,bf16}.hip and, with a float residual stream, tk_rows_{f16,bf16}_r32.hip; the
// C entry points are in tk_rows.hip.
//
// All of them are bound by memory, and are not far from being bound by their instructions: 4 to 20
// bytes an element for 15 to 40 vector instructions.
// Bytes that must move over the time that was measured, on MI355X (streams of this size reach
// 6.5 TB/s): dropout-add bf16 8192x4096 6.2 TB/s, its backward 5.5; layer norm bf16 16384x8192
// with a float stream 6.2, its backward 16384x4096 5.5; fused forward bf16 16384x8192 5.9, fused
// backward 8192x8192 5.6.
//
// A lane handles chunks of CH consecutive elements of a row: 16 bytes of the wider of the two
// types.  Addresses need only element alignment (gfx950 takes vector loads and stores at any),
// so odd widths and row pitches run the same code.  A row's last chunk may reach past its end:
// it is loaded from the row's last CH elements, unconditionally like every other chunk, and
// shifted into place when it is used; its stores go element by element.  Rows of fewer than
// CH elements run the kernels with CH = 1, where no chunk is partial.
#pragma once

#include <type_traits>

#include "tk_device_api.h"
#include "tk_rows_args.h"

namespace tk {

typedef _Float16 f16_t;
typedef __bf16 bf16_t;

template <class T, class R>
constexpr int kChunk = 16 / (sizeof(T) > sizeof(R) ? (int)sizeof(T) : (int)sizeof(R));

// ---- chunks ----------------------------------------------------------------------------
template <class T, int CH>
using Chunk = T __attribute__((ext_vector_type(CH), aligned(sizeof(T))));

// Where the chunk at column c is loaded from: the row's last CH elements if it reaches past the
// end (columns beyond the row too: what they load is not used).
template <int CH, class N>
__device__ __forceinline__ N chunk_at(N c, N cols) {
  return c + CH <= cols ? c : cols - CH;
}

// kOnce: past the caches.  Calls that read up to kCachedReads use ordinary loads: what a call of
// that size reads was often written just before and still lies in the 256 MB last-level cache.
// MI355X, calls in a row over three sets of buffers, ordinary against non-temporal loads:
// layer norm bf16 16384x1024 (reads 34 MB) 12.3 against 13.9 us, 262144x128 (67 MB) 21.6
// against 24.9, dropout-add's backward 8192x4096 (67 MB) 25.6 against 30.4; dropout-add
// 8192x4096 (134 MB) 38.4 against 36.8, layer norm 16384x8192 with a float stream (537 MB)
// 143 against 131, the fused backward 8192x8192 (403 MB) 137 against 131.
template <bool kOnce, int CH, class T>
__device__ __forceinline__ Chunk<T, CH> load_chunk(const T *p) {
  return kOnce ? __builtin_nontemporal_load((const Chunk<T, CH> *)p) : *(const Chunk<T, CH> *)p;
}

// The elements of a loaded chunk as floats, of which the first nv count; the rest become 0.
template <int CH, class T>
__device__ __forceinline__ void unpack(const Chunk<T, CH> &t, int nv, float *v) {
#pragma unroll
  for (int e = 0; e < CH; ++e) v[e] = (float)t[e];
  if (nv < CH) {
    const int down = nv > 0 ? CH - nv : CH;
#pragma unroll
    for (int step = CH; step; step >>= 1)
      if (down & step)
#pragma unroll
        for (int e = 0; e < CH; ++e) v[e] = e + step < CH ? v[e + step] : 0.0f;
  }
}

template <int CH, class T>
__device__ __forceinline__ void store_chunk(T *p, int nv, const float *v) {
  if (nv >= CH) {
    Chunk<T, CH> t;
#pragma unroll
    for (int e = 0; e < CH; ++e) t[e] = (T)v[e];  // to nearest even
    __builtin_nontemporal_store(t, (Chunk<T, CH> *)p);
  } else {
#pragma unroll
    for (int e = 0; e < CH; ++e)
      if (e < nv) p[e] = (T)v[e];
  }
}

// A parameter vector's chunk at column c: float or T elements, `other` where there is none.
template <int CH, class T>
__device__ __forceinline__ void load_param(const void *p, bool f32, uint32_t c, uint32_t cols, float other, float *v) {
  const uint32_t at = chunk_at<CH>(c, cols);
  const int nv = (int)(cols - c);
  if (!p) {
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] = other;
  } else if (f32) {
    unpack<CH, float>(*(const Chunk<float, CH> *)((const float *)p + at), nv, v);
  } else {
    unpack<CH, T>(*(const Chunk<T, CH> *)((const T *)p + at), nv, v);
  }
}

// ---- dropout ---------------------------------------------------------------------------
// Kept values over 1 - p: the IEEE quotient for float, and for the 16-bit types a product with the
// reciprocal as two floats, rounded once: within 2^-46 of the quotient before that rounding, so the
// same float but for a few in 10^7 (with the reciprocal rounded to float a quarter of all are
// others).  Their residual stream, statistics and the bias's gradient may be float, and all
// calls of one mask are to agree, so every one takes both products: up to 2 % of a
// backward (dropout-add 8192x4096 without bias 20.9 -> 21.3 us), nothing forward.
template <bool kDivide>
__device__ __forceinline__ float over_q(const Drop &d, float v) {
  return kDivide ? __fdiv_rn(v, d.q) : __builtin_fmaf(v, d.rq, v * d.rl);
}

// The words of a chunk whose first counter c is a multiple of CH share most of the hash's first
// step: with k = c ^ hk ^ ((c ^ hk) >> 16), the argument of the first product for counter c + j
// is k ^ j (j < CH changes no higher bit), and (k ^ j) K = k K + the sum over the bits b of j of
// +-2^b K, + where k's bit b is clear.  One product and CH - 1 additions instead of CH products,
// which take four cycles each: 14 instead of 18 cycles an element in all.
constexpr uint32_t kHashMul1 = 0x7FEB352Du, kHashMul2 = 0x846CA68Bu;  // tk_hash32's

// The product does not wait for the hash; the choice comes last.
template <bool kDivide>
__device__ __forceinline__ float drop_one(const Drop &d, uint32_t word, float v) {
  const bool keep = (word & 0x7FFFFFu) >= d.threshold;
  return keep ? over_q<kDivide>(d, v) : 0.0f;
}

template <bool kDivide, int CH>
__device__ __forceinline__ void drop_chunk(const Drop &d, uint32_t c, float *v) {
  if (CH > 1 && (c & (CH - 1)) == 0) {
    uint32_t k = c ^ d.hk;
    k ^= k >> 16;
    uint32_t x[CH];
    x[0] = k * kHashMul1;
#pragma unroll
    for (int b = 1; b < CH; b <<= 1) {
      const uint32_t step = k & b ? 0u - b * kHashMul1 : b * kHashMul1;
#pragma unroll
      for (int e = 0; e < b; ++e) x[b + e] = x[e] + step;
    }
#pragma unroll
    for (int e = 0; e < CH; ++e) {
      const uint32_t y = (x[e] ^ (x[e] >> 15)) * kHashMul2;
      v[e] = drop_one<kDivide>(d, y ^ (y >> 16), v[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] = drop_one<kDivide>(d, tk_word(d.hk, c + e), v[e]);
  }
}

// ---- sums over a row's lanes -----------------------------------------------------------
template <int kCtrl>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), kCtrl, 0xF, 0xF, true));
}

// Sums over pairs of lanes 16 and 32 apart: the row swaps of gfx950.
__device__ __forceinline__ float swap_sum16(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
__device__ __forceinline__ float swap_sum32(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// The sum over each group of kLanes lanes (a power of two), the same bits in all of them:
// pairs, quads, then mirrored halves within 16 lanes, then the row swaps of gfx950.
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float x) {
  if (kLanes >= 2) x += dpp<0xB1>(x);    // quad_perm 1,0,3,2
  if (kLanes >= 4) x += dpp<0x4E>(x);    // quad_perm 2,3,0,1
  if (kLanes >= 8) x += dpp<0x141>(x);   // row_half_mirror
  if (kLanes >= 16) x += dpp<0x140>(x);  // row_mirror
  if (kLanes >= 32) x = swap_sum16(x);
  if (kLanes >= 64) x = swap_sum32(x);
  return x;
}

// The sum over a wave's groups of kLanes lanes, lane by lane of a group.
template <int kLanes>
__device__ __forceinline__ float groups_sum(float x) {
  if (kLanes <= 8) x += dpp<0x128>(x);  // row_ror:8
  if (kLanes <= 16) x = swap_sum16(x);
  if (kLanes <= 32) x = swap_sum32(x);
  return x;
}

// How a work-group's threads take rows: kLanes (8, 16 or 32) lanes to a row, two waves (128,
// forward), or with kLanes = 64 as many whole waves (1 to 16) as the row needs, `waves`.  Whole
// waves keep the row and its addresses on the scalar unit.
template <int kLanes>
struct Team {
  uint32_t group, t, threads, groups;  // this thread's row group and place in it; a group's threads; groups
  __device__ __forceinline__ explicit Team(uint32_t waves) {
    if constexpr (kLanes < 64) {
      group = threadIdx.x / kLanes;
      t = threadIdx.x % kLanes;
      threads = kLanes;
    } else {
      if (kLanes == 128) waves = 2;
      group = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / waves;
      threads = waves * 64;
      t = threadIdx.x - group * threads;
    }
    groups = blockDim.x / threads;
  }
};

// kN sums over a row.  Rows of up to a wave stay in registers; wider ones go through `slot` (kN
// floats a wave of the work-group), which must not be written again before another barrier has
// passed: every lane reads one wave's sums and the lanes add them up.
template <int kLanes, int kN>
__device__ __forceinline__ void row_sums(float (&x)[kN], float (*slot)[kN], uint32_t group, uint32_t waves) {
#pragma unroll
  for (int k = 0; k < kN; ++k) x[k] = lanes_sum<kLanes>(x[k]);
  if (kLanes == 64 && waves > 1) {
    const uint32_t lane = threadIdx.x & 15;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < kN; ++k) slot[threadIdx.x >> 6][k] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kN; ++k) x[k] = lanes_sum<16>(lane < waves ? slot[group * waves + lane][k] : 0.0f);
  }
}

// The forward kernels' sum over a row, like row_sums.  kLanes = 128: `other` gets the sum over the
// work-group's other row (elsewhere 0).
template <int kLanes>
__device__ __forceinline__ float row_sum(float x, float *slot, uint32_t group, uint32_t waves, float &other) {
  other = 0.0f;
  x = lanes_sum<kLanes < 64 ? kLanes : 64>(x);
  if (kLanes < 64 || (kLanes == 64 && waves == 1)) return x;
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = x;
  __syncthreads();
  if (kLanes == 128) {
    const float y = lanes_sum<2>(slot[(group * 2 + (threadIdx.x & 3)) & 3]);  // lanes 0 and 1 this row's, 2 and 3 the other's
    other = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(y), 2));
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(y), 0));
  }
  const uint32_t lane = threadIdx.x & 15;
  return lanes_sum<16>(lane < waves ? slot[group * waves + lane] : 0.0f);
}

// ---- forward ---------------------------------------------------------------------------
// A chunk of a row's inputs as loaded.
template <class T, class R, bool kX, bool kOnce, int CH>
struct FwdIn {
  Chunk<T, CH> x;
  Chunk<R, CH> r;
  __device__ __forceinline__ void load(const FwdArgs &a, uint64_t row, uint32_t c) {
    const uint32_t at = chunk_at<CH>(c, a.cols);
    if constexpr (kX) x = load_chunk<kOnce, CH>((const T *)a.x + row * a.ldx + at);
    if (!kX || a.residual) r = load_chunk<kOnce, CH>((const R *)a.residual + row * a.ldr + at);
  }
  // The norm's input: residual + drop(x + bias); 0 past the row's end.
  __device__ __forceinline__ void value(const FwdArgs &a, uint64_t row, uint32_t c, const float *bias, float *v) const {
    const int nv = (int)(a.cols - c);
    if constexpr (kX) {
      unpack<CH, T>(x, nv, v);
      if (a.bias)
#pragma unroll
        for (int e = 0; e < CH; ++e) v[e] += bias[e];
      if (a.drop.on) drop_chunk<std::is_same<T, float>::value, CH>(a.drop, a.drop.start + (uint32_t)row * a.cols + c, v);
      if (a.residual) {
        float u[CH];
        unpack<CH, R>(r, nv, u);
#pragma unroll
        for (int e = 0; e < CH; ++e) v[e] += u[e];
      }
    } else {
      unpack<CH, R>(r, nv, v);
    }
  }
};

// y from the distances d of a chunk's elements to the row's mean.
template <class T, int CH>
__device__ __forceinline__ void norm_out(const FwdArgs &a, uint64_t row, uint32_t c, float rstd, const float *gamma,
                                         const float *beta, const float *d) {
  const int nv = (int)(a.cols - c);
  if (nv <= 0) return;
  float y[CH];
#pragma unroll
  for (int e = 0; e < CH; ++e) y[e] = __builtin_fmaf(d[e] * rstd, gamma[e], beta[e]);
  store_chunk<CH>((T *)a.y + row * a.ldy + c, nv, y);
}

// 1 / sqrt(x) to within two units of the last place: the hardware's v_rsq_f32 (one unit), with
// the argument scaled into its range where it might be subnormal (eps = 0).
__device__ __forceinline__ float rsqrt_any(float x) {
  return x < 0x1p-96f ? __builtin_amdgcn_rsqf(x * 0x1p96f) * 0x1p48f : __builtin_amdgcn_rsqf(x);
}

// Whether a row's mean is more than four standard deviations from zero.  It is corrected then: the
// sum's rounding makes it some units of its last place wrong, no small part of a distance from it
// (rows of 10000.1 in f32: h = -0.3 to -0.8 where it is 0), but the distances themselves are
// nearly exact, and their own mean is what it is off by.  Nearer to zero their sum is no more exact
// than the first one (layer norm bf16 16384x8192, float stream, mean 0: the mean's relative error
// is 1.1e-7, corrected 7.6e-7).  Only such rows pay for one sum more: with the sum of the distances
// in every row, layer norm bf16 16384x4096, which is bound by its instructions, took 51 us for 46.
// Never true of sums beyond f32 or NaN; where it is true, all that follows is finite.
__device__ __forceinline__ bool far_from_zero(float mean, float m2, float inv) { return mean * mean > m2 * inv * 16.0f; }

// A sum over the columns divided by them, rounded once but for rare cases: the product with the
// rounded reciprocal and one step of Newton's.  An exact quotient comes out exact, so that the
// distances of a constant row end as zeros.
__device__ __forceinline__ float mean_of(float sum, uint32_t n, float inv) {
  __asm__ volatile("" : "+s"(n));  // converted here, not kept in a register between rows
  const float cols = (float)n, q = sum * inv;
  return __builtin_fmaf(__builtin_fmaf(-q, cols, sum), inv, q);
}

// The sum of squared distances to a mean that is `delta` higher: `off` is the distances' own sum.
// The difference is some squared roundings of the mean (never below 0 but for its own rounding).
__device__ __forceinline__ float squares_about(float m2, float off, float delta) {
  return fmaxf(__builtin_fmaf(-off, delta, m2), 0.0f);
}

// The row stays in registers between the two sums (the mean, then the squared distances from
// it: no cancellation) and the output: one read and one write of the data.  A work-group takes
// every gridDim.x-th set of rows, keeps the parameters in registers, and loads its next rows
// before it works on the present ones.
template <class T, class R, bool kX, bool kOnce, int CH, int kLanes, int V, bool kKeep>
__global__ __launch_bounds__(kLanes == 64 ? 1024 : 256) void k_norm_fwd(FwdArgs a) {
  __shared__ float slot[3][16];  // one for each sum: a barrier lies between a slot's use and its next
  Team<kLanes> team(a.waves);
  const uint64_t step = (uint64_t)gridDim.x * team.groups;
  uint64_t base = (uint64_t)blockIdx.x * team.groups, row = base + team.group;
  float bias[kKeep ? V : 1][CH], gamma[kKeep ? V : 1][CH], beta[kKeep ? V : 1][CH];
  FwdIn<T, R, kX, kOnce, CH> next[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t c = (j * team.threads + team.t) * CH;
    if (row < a.rows) next[j].load(a, row, c);
    if constexpr (kKeep) {
      if (kX) load_param<CH, T>(a.bias, a.params_f32, c, a.cols, 0.0f, bias[j]);
      load_param<CH, T>(a.gamma, a.params_f32, c, a.cols, 1.0f, gamma[j]);
      load_param<CH, T>(a.beta, a.params_f32, c, a.cols, 0.0f, beta[j]);
    }
  }
  const float inv = 1.0f / (float)a.cols;
  // every wave of a work-group runs the same rounds: the sums have barriers
  for (; base < a.rows; base += step, row += step) {
    if (V * CH > 8) __asm__ volatile("" : "+v"(team.t));  // addresses are made anew each round, not kept
    float v[V][CH], s = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t c = (j * team.threads + team.t) * CH;
      if (kX && !kKeep) load_param<CH, T>(a.bias, a.params_f32, c, a.cols, 0.0f, bias[0]);
      next[j].value(a, row, c, bias[kKeep ? j : 0], v[j]);
#pragma unroll
      for (int e = 0; e < CH; ++e) s += v[j][e];
      if (!kKeep) __builtin_amdgcn_sched_barrier(0);  // one chunk's temporaries at a time
    }
    if (row + step < a.rows)
#pragma unroll
      for (int j = 0; j < V; ++j) next[j].load(a, row + step, (j * team.threads + team.t) * CH);
    float s_other, m2_other, mean = row_sum<kLanes>(s, slot[0], team.group, a.waves, s_other) * inv, m2 = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t c = (j * team.threads + team.t) * CH;
      const int nv = (int)(a.cols - c);
      if (a.sum && nv > 0 && row < a.rows) store_chunk<CH>((R *)a.sum + row * a.lds + c, nv, v[j]);
#pragma unroll
      for (int e = 0; e < CH; ++e) v[j][e] -= mean;
      if (nv < CH)  // past the end: no distance from the mean
#pragma unroll
        for (int e = 0; e < CH; ++e) v[j][e] = e < nv ? v[j][e] : 0.0f;
#pragma unroll
      for (int e = 0; e < CH; ++e) m2 = __builtin_fmaf(v[j][e], v[j][e], m2);
    }
    m2 = row_sum<kLanes>(m2, slot[1], team.group, a.waves, m2_other);
    // The same bits, so the same answer, in all waves of a row; of two rows in a work-group either's:
    // its waves meet the barrier below together.
    const bool far = far_from_zero(mean, m2, inv);
    if (__any(far || (kLanes == 128 && far_from_zero(s_other * inv, m2_other, inv)))) {
      float off = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < CH; ++e) off += v[j][e];
      off = row_sum<kLanes>(off, slot[2], team.group, a.waves, s_other);
      const float delta = far ? mean_of(off, a.cols, inv) : 0.0f;  // of the wave's other rows: as it was
      mean = far ? mean + delta : mean;
      m2 = far ? squares_about(m2, off, delta) : m2;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < CH; ++e) v[j][e] -= delta;
    }
    const float rstd = rsqrt_any(__builtin_fmaf(m2, inv, a.eps));
    if (row < a.rows) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t c = (j * team.threads + team.t) * CH;
        if constexpr (!kKeep) {
          load_param<CH, T>(a.gamma, a.params_f32, c, a.cols, 1.0f, gamma[0]);
          load_param<CH, T>(a.beta, a.params_f32, c, a.cols, 0.0f, beta[0]);
        }
        norm_out<T, CH>(a, row, c, rstd, gamma[kKeep ? j : 0], beta[kKeep ? j : 0], v[j]);
        if (!kKeep) __builtin_amdgcn_sched_barrier(0);
      }
      if (team.t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
    }
  }
}

// Rows too wide for the registers of one work-group: the same sums over three passes (four far
// from zero), the inputs read again in each (a row of some hundred KB stays in the caches).
// Nothing is written before the last pass, and there each element's inputs are read by the
// thread that writes it, so outputs in place of inputs are fine.
template <class T, class R, bool kX>
__global__ __launch_bounds__(1024) void k_norm_fwd_wide(FwdArgs a) {
  constexpr int CH = kChunk<T, R>, kTpr = 1024;
  __shared__ float slot[3][kTpr / 64];
  const float inv = 1.0f / (float)a.cols;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const auto chunk = [&](uint32_t c, float *v) {
      FwdIn<T, R, kX, false, CH> in;
      float bias[CH];
      in.load(a, row, c);
      if (kX) load_param<CH, T>(a.bias, a.params_f32, c, a.cols, 0.0f, bias);
      in.value(a, row, c, bias, v);
    };
    float v[CH], s = 0.0f;
    for (uint32_t c = threadIdx.x * CH; c < a.cols; c += kTpr * CH) {
      chunk(c, v);
      const int nv = (int)(a.cols - c);
#pragma unroll
      for (int e = 0; e < CH; ++e) s += e < nv ? v[e] : 0.0f;
    }
    float other, mean = row_sum<64>(s, slot[0], 0, kTpr / 64, other) * inv, delta = 0.0f, m2 = 0.0f;
    for (uint32_t c = threadIdx.x * CH; c < a.cols; c += kTpr * CH) {
      chunk(c, v);
      const int nv = (int)(a.cols - c);
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        const float d = e < nv ? v[e] - mean : 0.0f;
        m2 = __builtin_fmaf(d, d, m2);
      }
    }
    m2 = row_sum<64>(m2, slot[1], 0, kTpr / 64, other);
    if (__any(far_from_zero(mean, m2, inv))) {  // the same in all waves
      s = 0.0f;
      for (uint32_t c = threadIdx.x * CH; c < a.cols; c += kTpr * CH) {
        chunk(c, v);
        const int nv = (int)(a.cols - c);
#pragma unroll
        for (int e = 0; e < CH; ++e) s += e < nv ? v[e] - mean : 0.0f;
      }
      s = row_sum<64>(s, slot[2], 0, kTpr / 64, other);
      delta = mean_of(s, a.cols, inv);
      m2 = squares_about(m2, s, delta);
    }
    const float rstd = rsqrt_any(__builtin_fmaf(m2, inv, a.eps));
    for (uint32_t c = threadIdx.x * CH; c < a.cols; c += kTpr * CH) {
      float gamma[CH], beta[CH];
      chunk(c, v);
      load_param<CH, T>(a.gamma, a.params_f32, c, a.cols, 1.0f, gamma);
      load_param<CH, T>(a.beta, a.params_f32, c, a.cols, 0.0f, beta);
      if (a.sum) store_chunk<CH>((R *)a.sum + row * a.lds + c, (int)(a.cols - c), v);
#pragma unroll
      for (int e = 0; e < CH; ++e) v[e] = v[e] - mean - delta;
      norm_out<T, CH>(a, row, c, rstd, gamma, beta, v);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean + delta;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// ---- backward --------------------------------------------------------------------------
// Layer norm's gradient for one element, rstd (g - mean(g) - h mean(g h)), with
// a = -rstd mean(g) and b = -rstd mean(g h).
__device__ __forceinline__ float norm_grad(float g, float h, float rstd, float a, float b) {
  return __builtin_fmaf(h, b, __builtin_fmaf(g, rstd, a));
}

// A chunk of a row's inputs as loaded.  dy is of type D: T, or R for dropout-add's gradient.
template <class T, class R, class D, bool kNorm, bool kOnce, int CH>
struct BwdIn {
  Chunk<D, CH> dy;
  Chunk<R, CH> sum, dsum;
  __device__ __forceinline__ void load(const BwdArgs &a, uint64_t row, uint32_t c) {
    const uint32_t at = chunk_at<CH>(c, a.cols);
    dy = load_chunk<kOnce, CH>((const D *)a.dy + row * a.lddy + at);
    if (kNorm) sum = load_chunk<kOnce, CH>((const R *)a.sum + row * a.lds + at);
    if (a.dsum) dsum = load_chunk<kOnce, CH>((const R *)a.dsum + row * a.ldds + at);
  }
  // h of every element
  __device__ __forceinline__ void normed(int nv, float mean, float rstd, float *h) const {
    unpack<CH, R>(sum, nv, h);
#pragma unroll
    for (int e = 0; e < CH; ++e) h[e] = (h[e] - mean) * rstd;
  }
  // Outputs: dresidual = v + dsum and dx = drop(dresidual), which comes back in v.
  template <bool kX>
  __device__ __forceinline__ void out(const BwdArgs &a, uint64_t row, uint32_t c, float *v) const {
    const int nv = (int)(a.cols - c);
    if (a.dsum) {
      float d[CH];
      unpack<CH, R>(dsum, nv, d);
#pragma unroll
      for (int e = 0; e < CH; ++e) v[e] += d[e];
    }
    if (a.dresidual) store_chunk<CH>((R *)a.dresidual + row * a.lddr + c, nv, v);
    if constexpr (kX) {
      if (a.drop.on) drop_chunk<std::is_same<T, float>::value, CH>(a.drop, a.drop.start + (uint32_t)row * a.cols + c, v);
      store_chunk<CH>((T *)a.dx + row * a.lddx + c, nv, v);
    }
  }
};

// Column sums of one work-group for all rows are the gradients themselves: element c of the
// k-th, rounded to the parameters' type.
template <class T>
__device__ __forceinline__ void put_gradient(const BwdArgs &a, int k, uint32_t c, float v) {
  if (!a.sums[k]) return;
  if (a.params_f32) ((float *)a.sums[k])[c] = v;
  else ((T *)a.sums[k])[c] = (T)v;
}

// The first nv of a chunk's sums to p, whole vectors where they fit.
template <int CH>
__device__ __forceinline__ void put_sums(float *p, int nv, const float *v, bool past = false) {
  if (nv >= CH) {
    Chunk<float, CH> t;
#pragma unroll
    for (int e = 0; e < CH; ++e) t[e] = v[e];
    if (past) {
      asm volatile("");  // the compiler makes one plain store of the two if it can
      __builtin_nontemporal_store(t, (Chunk<float, CH> *)p);
      asm volatile("");
    } else {
      *(Chunk<float, CH> *)p = t;
    }
  } else {
#pragma unroll
    for (int e = 0; e < CH; ++e)
      if (e < nv) p[e] = v[e];
  }
}

// Rows in registers, as forward: as loaded, between the sums and the output.  A work-group
// takes every gridDim.x-th set of rows and keeps the column sums of its own rows in registers;
// at the end its groups' sums are added up through LDS and written to the workspace, one line
// of partial sums per work-group, which k_finish adds up in order.  Sixteen waves have 128
// registers; with three sums, the f32 kernels and those of whole waves with a float stream spill 2
// (9 with 32 lanes to a row), 12 to 16 bytes a lane.
template <class T, class R, bool kX, bool kBias, bool kOnce, int CH, int kLanes, int V>
__global__ __launch_bounds__(1024) void k_norm_bwd(BwdArgs a) {
  constexpr int kSums = kBias ? 3 : 2;
  __shared__ float slot[2][16][2];
  const Team<kLanes> team(a.waves);
  const uint64_t step = (uint64_t)gridDim.x * team.groups;
  uint64_t base = (uint64_t)blockIdx.x * team.groups, row = base + team.group;
  const float inv = 1.0f / (float)a.cols;
  float acc[kSums][V][CH], gamma[V][CH], mean = 0.0f, rstd = 0.0f;
  BwdIn<T, R, T, true, kOnce, CH> next[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t c = (j * team.threads + team.t) * CH;
    if (row < a.rows) next[j].load(a, row, c);
    load_param<CH, T>(a.gamma, a.params_f32, c, a.cols, 1.0f, gamma[j]);
#pragma unroll
    for (int k = 0; k < kSums; ++k)
#pragma unroll
      for (int e = 0; e < CH; ++e) acc[k][j][e] = 0.0f;
  }
  if (row < a.rows) {
    mean = a.mean[row];
    rstd = a.rstd[row];
  }
  int par = 0;  // the slot in use: one barrier a round keeps the other one safe to write
  for (; base < a.rows; base += step, row += step, par ^= 1) {
    const bool here = row < a.rows;
    const float m = mean, rs = rstd;
    BwdIn<T, R, T, true, kOnce, CH> in[V];
#pragma unroll
    for (int j = 0; j < V; ++j) in[j] = next[j];
    if (row + step < a.rows) {
#pragma unroll
      for (int j = 0; j < V; ++j) next[j].load(a, row + step, (j * team.threads + team.t) * CH);
      mean = a.mean[row + step];
      rstd = a.rstd[row + step];
    }
    float g[V][CH], h[V][CH], s[2] = {0.0f, 0.0f};
    if (here) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int nv = (int)(a.cols - (j * team.threads + team.t) * CH);
        unpack<CH, T>(in[j].dy, nv, g[j]);
        in[j].normed(nv, m, rs, h[j]);
#pragma unroll
        for (int e = 0; e < CH; ++e) {
          acc[0][j][e] = __builtin_fmaf(g[j][e], h[j][e], acc[0][j][e]);
          acc[1][j][e] += g[j][e];
          g[j][e] *= gamma[j][e];
          s[0] += g[j][e];
          s[1] = __builtin_fmaf(g[j][e], h[j][e], s[1]);
        }
      }
    }
    row_sums<kLanes>(s, slot[par], team.group, a.waves);
    const float ka = -rs * (s[0] * inv), kb = -rs * (s[1] * inv);
    if (here) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t c = (j * team.threads + team.t) * CH;
#pragma unroll
        for (int e = 0; e < CH; ++e) g[j][e] = norm_grad(g[j][e], h[j][e], rs, ka, kb);
        in[j].template out<kX>(a, row, c, g[j]);
        if constexpr (kBias) {
#pragma unroll
          for (int e = 0; e < CH; ++e) acc[2][j][e] += g[j][e];
        }
      }
    }
  }
  if (!a.partial && !a.alone) return;
  // The groups' sums of the same columns: first over the groups of a wave, in registers, then
  // over the waves, one vector at a time through (dynamic) LDS.  A group alone writes its
  // registers: through LDS, 32x8192 takes 10.5 us for 8.0.
  constexpr uint32_t kWaveCols = (kLanes < 64 ? kLanes : 64) * V * CH;
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, waves = kLanes < 64 ? 1 : a.waves;
  const uint32_t groups = (blockDim.x >> 6) / waves;
  extern __shared__ __align__(16) float tile[];
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
    float *line = a.partial + ((uint64_t)k * gridDim.x + blockIdx.x) * line_pitch(a.cols);
    if (groups > 1 || a.alone) {
      if (k) __syncthreads();
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < CH; ++e) acc[k][j][e] = groups_sum<kLanes>(acc[k][j][e]);
      if (lane < kLanes)
#pragma unroll
        for (int j = 0; j < V; ++j)
          put_sums<CH>(tile + wave / waves * (waves * kWaveCols) + (j * team.threads + team.t) * CH, CH, acc[k][j]);
      __syncthreads();
      const auto sums = [&](auto put) {
        for (uint32_t c = threadIdx.x; c < a.cols; c += blockDim.x) {
          float s = 0.0f;
#pragma unroll 8
          for (uint32_t r = 0; r < groups; ++r) s += tile[r * (waves * kWaveCols) + c];
          put(c, s);
        }
      };
      if (a.alone) sums([&](uint32_t c, float s) { put_gradient<T>(a, k, c, s); });
      else if (a.past) sums([&](uint32_t c, float s) { __builtin_nontemporal_store(s, line + c); });
      else sums([&](uint32_t c, float s) { line[c] = s; });
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t c = (j * team.threads + team.t) * CH;
        put_sums<CH>(line + c, (int)(a.cols - c), acc[k][j], a.past);
      }
    }
  }
}

// Rows wider than k_norm_bwd's registers hold with their column sums: first norm_grad's two
// numbers for every row, then k_cols_bwd over columns, which reads dy and sum again (here they
// are read through the caches).
template <class T, class R>
__global__ __launch_bounds__(1024) void k_row_stats(BwdArgs a) {
  constexpr int CH = kChunk<T, R>, kTpr = 1024;
  __shared__ float slot[2][kTpr / 64][2];
  int par = 0;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, par ^= 1) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s[2] = {0.0f, 0.0f};
    const T *dy = (const T *)a.dy + row * a.lddy;
    const R *sum = (const R *)a.sum + row * a.lds;
    uint32_t c = threadIdx.x * CH;
    // the next chunk is loaded before the present one is used (past the end: the row's last, unused)
    Chunk<T, CH> next_dy = load_chunk<false, CH>(dy + chunk_at<CH>(c, a.cols));
    Chunk<R, CH> next_sum = load_chunk<false, CH>(sum + chunk_at<CH>(c, a.cols));
    for (; c < a.cols; c += kTpr * CH) {
      const int nv = (int)(a.cols - c);
      const uint32_t at = chunk_at<CH>(c + kTpr * CH, a.cols);
      float g[CH], h[CH], w[CH];
      const Chunk<T, CH> here_dy = next_dy;
      const Chunk<R, CH> here_sum = next_sum;
      next_dy = load_chunk<false, CH>(dy + at);
      next_sum = load_chunk<false, CH>(sum + at);
      load_param<CH, T>(a.gamma, a.params_f32, c, a.cols, 1.0f, w);
      unpack<CH, T>(here_dy, nv, g);
      unpack<CH, R>(here_sum, nv, h);
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        const float x = g[e] * w[e];
        s[0] += x;
        s[1] = __builtin_fmaf(x, (h[e] - mean) * rstd, s[1]);
      }
    }
    row_sums<64>(s, slot[par], 0, kTpr / 64);
    if (threadIdx.x == 0) {
      a.stats[2 * row] = -rstd * (s[0] / (float)a.cols);
      a.stats[2 * row + 1] = -rstd * (s[1] / (float)a.cols);
    }
  }
}

// A strip of kLanes lanes' chunks, 64 / kLanes rows to each of sixteen waves at a time, the next
// ones prefetched: each lane keeps the sums of its own columns.  kNorm: layer norm's gradient
// with the rows' numbers from k_row_stats; else dy (of the residual stream's type) is the sum's
// gradient itself.
//
// The work-groups of a strip take every gridDim.y-th set of rows, so that all of them together
// are within some MB at any time (ranges of rows, with powers of two between them, took 26 to 39
// us for dropout-add's backward bf16 8192x4096, by where the buffers lay).  Sixteen waves to a
// work-group keep the lines of partial sums few: 32768x512 takes 14.7 us, with four waves and
// 2048 lines 20.5; 65536x64, eight rows to a wave, 7.4 us, with one row to a wave 24.
template <class T, class R, bool kNorm, bool kX, bool kBias, bool kOnce, int CH, int kLanes>
__global__ __launch_bounds__(1024) void k_cols_bwd(BwdArgs a) {
  constexpr int kSums = (kNorm ? 2 : 0) + (kBias ? 1 : 0), kGroups = 64 / kLanes;
  typedef typename std::conditional<kNorm, T, R>::type D;
  const uint32_t lane = threadIdx.x & 63, wave = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t strip = a.strip0 + blockIdx.x, c = (strip * kLanes + lane % kLanes) * CH;
  const int nv = (int)(a.cols - c);
  const uint64_t step = (uint64_t)gridDim.y * (16 * kGroups);
  float acc[kSums ? kSums : 1][CH];
#pragma unroll
  for (int k = 0; k < kSums; ++k)
#pragma unroll
    for (int e = 0; e < CH; ++e) acc[k][e] = 0.0f;
  if (nv > 0) {
    float w[CH];
    if (kNorm) load_param<CH, T>(a.gamma, a.params_f32, c, a.cols, 1.0f, w);
    BwdIn<T, R, D, kNorm, kOnce, CH> next;
    uint64_t row = ((uint64_t)blockIdx.y * 16 + wave) * kGroups + (kGroups > 1 ? lane / kLanes : 0);
    if (row < a.rows) next.load(a, row, c);
    for (; row < a.rows; row += step) {
      const BwdIn<T, R, D, kNorm, kOnce, CH> in = next;
      if (row + step < a.rows) next.load(a, row + step, c);
      float v[CH];
      unpack<CH, D>(in.dy, nv, v);
      if constexpr (kNorm) {
        const float rstd = a.rstd[row], ka = a.stats[2 * row], kb = a.stats[2 * row + 1];
        float h[CH];
        in.normed(nv, a.mean[row], rstd, h);
#pragma unroll
        for (int e = 0; e < CH; ++e) {
          acc[0][e] = __builtin_fmaf(v[e], h[e], acc[0][e]);
          acc[1][e] += v[e];
          v[e] = norm_grad(v[e] * w[e], h[e], rstd, ka, kb);
        }
      }
      in.template out<kX>(a, row, c, v);
      if constexpr (kBias) {
#pragma unroll
        for (int e = 0; e < CH; ++e) acc[kSums - 1][e] += v[e];
      }
    }
  }
  if constexpr (kSums > 0) {
    if (!a.partial && !a.alone) return;
    __shared__ __align__(16) float tile[16][kLanes * CH];
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
      if (k) __syncthreads();
#pragma unroll
      for (int e = 0; e < CH; ++e) acc[k][e] = groups_sum<kLanes>(acc[k][e]);
      if (lane < kLanes) put_sums<CH>(tile[wave] + lane * CH, CH, acc[k]);
      __syncthreads();
      float *line = a.partial + ((uint64_t)k * gridDim.y + blockIdx.y) * line_pitch(a.cols);
      const uint32_t i = threadIdx.x, col = strip * (kLanes * CH) + i;
      if (i < kLanes * CH && col < a.cols) {
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) s += tile[r][i];
        if (a.alone) put_gradient<T>(a, kNorm ? k : 2, col, s);
        else line[col] = s;
      }
    }
  }
}

// ---- dropout-add, element by element ---------------------------------------------------
// Chunk n of the call lies in row n / chunks_per_row.  A work-group's first row is found on the
// scalar unit and its lanes' rows from there, a few rows further: one product a matrix.  The
// quotient is a product with the rounded-up reciprocal: exact below 2^31 chunks, which a launch
// stays under.
__device__ __forceinline__ uint32_t row_of(const AddArgs &a, uint32_t n) {
  return a.div_shift < 0 ? n : __umulhi(n, a.div_mul) >> a.div_shift;
}

template <class TI, class TO, bool kDivide, bool kOnce, bool kFlat, int CH, class TP>
__global__ __launch_bounds__(256) void k_drop_add(AddArgs a) {
  const uint32_t first = blockIdx.x * 256u;
  uint32_t dr = 0, column = 0;  // rows from the work-group's first, chunks from the row's start
  uint64_t row0 = 0;
  if (!kFlat || a.bias) {
    const uint32_t r0 = row_of(a, first), n = first - r0 * a.chunks_per_row + threadIdx.x;  // from that row's start
    dr = row_of(a, n);
    column = n - dr * a.chunks_per_row;
    row0 = a.row0 + r0;
  }
  if (first + threadIdx.x >= a.chunks) return;
  const uint64_t c = (uint64_t)(kFlat ? first + threadIdx.x : column) * CH, from = chunk_at<CH>(c, a.cols64);
  const auto at = [&](uint64_t ld, uint64_t k) { return kFlat ? k : row0 * ld + ((uint64_t)dr * (uint32_t)ld + k); };
  const Chunk<TI, CH> x = load_chunk<kOnce, CH>((const TI *)a.x + at(a.ldx, from));
  Chunk<TO, CH> d;
  if (a.residual) d = load_chunk<kOnce, CH>((const TO *)a.residual + at(a.ldr, from));
  const int nv = a.cols64 - c < CH ? (int)(a.cols64 - c) : CH;
  float v[CH], b[CH];
  if (a.bias) load_param<CH, TP>(a.bias, a.params_f32, column * CH, (uint32_t)a.bias_cols, 0.0f, b);
  unpack<CH, TI>(x, nv, v);
  if (a.bias)
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] += b[e];
  if (a.drop.on) drop_chunk<kDivide, CH>(a.drop, a.drop.start + (uint32_t)at(a.cols64, c), v);
  if (a.residual) {
    float t[CH];
    unpack<CH, TO>(d, nv, t);
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] += t[e];
  }
  store_chunk<CH>((TO *)a.y + at(a.ldy, c), nv, v);
}

// ---- launches --------------------------------------------------------------------------
// Work-groups over sets of rows; the kernels loop beyond.
static inline uint32_t row_grid(uint64_t sets, uint32_t most) { return (uint32_t)(sets < most ? sets : most); }

// A grid that the device holds at once, each set of rows prefetched: up to 20 waves a compute
// unit with eight elements a lane (80 registers), 24 where that makes two work-groups of one,
// and 16 with more elements (128 registers).  Layer norm bf16 32768x2048 takes 61, 49, 46, 45,
// 48 and 55 us with 8, 12, 16, 20, 24 and 32 waves, and 71 us with a work-group for each row
// and no prefetch; the fused forward 8192x4096 49 to 53, and 62.  The fused forward with a float
// stream has 84 registers, five waves to a SIMD: it stays at 20 waves (bf16 512x6144 9.6 us, with
// two work-groups of twelve, half of which wait, 12.7; 8192x6144 102 and 106).
template <class T, class R, bool kX, bool kOnce, int CH, int kLanes, int V, bool kKeep = true>
static void launch_fwd(FwdArgs a, hipStream_t s) {
  constexpr uint32_t kCols = kLanes * V * CH;
  a.waves = kLanes < 64 ? 1 : kLanes == 128 ? 2 : (a.cols + kCols - 1) / kCols;
  const uint32_t waves = a.waves >= 4 ? a.waves : 4 / a.waves * a.waves;  // of a work-group
  const uint32_t rows = kLanes < 64 ? 64 * waves / kLanes : waves / a.waves;
  constexpr bool kMixed = kX && !std::is_same<T, R>::value;
  const uint32_t each = (V * CH > 8 ? 16 : waves > 8 && !kMixed ? 24 : 20) / waves;  // work-groups of a compute unit
  hipLaunchKernelGGL((k_norm_fwd<T, R, kX, kOnce, CH, kLanes, V, kKeep>),
                     dim3(row_grid((a.rows + rows - 1) / rows, 256 * (each ? each : 1))), dim3(64 * waves), 0, s, a);
}

// Lanes to a row by its width, eight elements a lane.  Beyond twelve waves a row (6144 columns)
// a lane takes sixteen, so that two rows share a compute unit (layer norm bf16 8192x8192 45.5
// against 53 us), and beyond sixteen waves of those 24 or 32, with the parameters read again for
// every row (fused forward bf16 1024x32768 59 us, in three passes 118; 655x20000 27 us with 24,
// 31 with 32; 4096x12288 71 us with sixteen and the parameters kept, 81 with 24).  The fused
// kernels with 32 elements a lane spill in f32 (50 registers) and with a float stream (26), and are
// faster all the same: f32 1024x32768 146 us, in three passes 172; bf16 with a float
// stream 102 and 147, 8x24577 16.9 and 20.2.
template <class T, class R, bool kX, bool kOnce>
static void norm_fwd_of(const FwdArgs &a, hipStream_t s) {
  constexpr int CH = kChunk<T, R>, K = 8 / CH;
  if (a.cols < CH) launch_fwd<T, R, kX, kOnce, 1, 8, 1>(a, s);
  else if (a.cols <= 64) launch_fwd<T, R, kX, kOnce, CH, 8, K>(a, s);
  else if (a.cols <= 128) launch_fwd<T, R, kX, kOnce, CH, 16, K>(a, s);
  else if (a.cols <= 256) launch_fwd<T, R, kX, kOnce, CH, 32, K>(a, s);
  else if (a.cols > 512 && a.cols <= 1024) launch_fwd<T, R, kX, kOnce, CH, 128, K>(a, s);
  else if (a.cols <= 6144) launch_fwd<T, R, kX, kOnce, CH, 64, K>(a, s);
  else if (a.cols <= 16384) launch_fwd<T, R, kX, kOnce, CH, 64, 2 * K>(a, s);
  else if (a.cols <= 24576) launch_fwd<T, R, kX, kOnce, CH, 64, 3 * K, false>(a, s);
  else if (a.cols <= 32768) launch_fwd<T, R, kX, kOnce, CH, 64, 4 * K, false>(a, s);
  else hipLaunchKernelGGL((k_norm_fwd_wide<T, R, kX>), dim3(row_grid(a.rows, 1u << 16)), dim3(1024), 0, s, a);
}

template <class T, class R, bool kX, bool kBias, bool kOnce, int CH, int kLanes, int V>
static void launch_bwd(const BwdArgs &a, const BwdPlan &p, hipStream_t s) {
  const uint32_t lds = (uint32_t)p.waves * kLanes * V * CH * 4;
  hipLaunchKernelGGL((k_norm_bwd<T, R, kX, kBias, kOnce, CH, kLanes, V>), dim3((uint32_t)p.lines), dim3(64 * p.waves), lds, s,
                     a);
}

template <class T, class R, bool kX, bool kBias, bool kOnce>
static void norm_bwd_as(const BwdArgs &a, const BwdPlan &p, hipStream_t s) {
  constexpr int CH = kChunk<T, R>, K = 8 / CH;
  if (a.cols < CH) launch_bwd<T, R, kX, kBias, kOnce, 1, 8, 1>(a, p, s);
  else if (p.lanes == 8) launch_bwd<T, R, kX, kBias, kOnce, CH, 8, K>(a, p, s);
  else if (p.lanes == 16) launch_bwd<T, R, kX, kBias, kOnce, CH, 16, K>(a, p, s);
  else if (p.lanes == 32) launch_bwd<T, R, kX, kBias, kOnce, CH, 32, K>(a, p, s);
  else launch_bwd<T, R, kX, kBias, kOnce, CH, 64, K>(a, p, s);
}

template <class T, class R, bool kNorm, bool kX, bool kBias, bool kOnce, int CH, int kLanes>
static void launch_cols(const BwdArgs &a, const BwdPlan &p, hipStream_t s) {
  // a launch holds fewer than 2^32 threads to a dimension
  constexpr uint64_t kMost = 1u << 20;
  BwdArgs b = a;
  for (uint64_t strip = 0; strip < p.strips; strip += kMost) {
    b.strip0 = (uint32_t)strip;
    hipLaunchKernelGGL((k_cols_bwd<T, R, kNorm, kX, kBias, kOnce, CH, kLanes>),
                       dim3((uint32_t)(p.strips - strip < kMost ? p.strips - strip : kMost), (uint32_t)p.lines), dim3(1024), 0,
                       s, b);
  }
}

template <class T, class R, bool kOnce>
static void add_bwd_as(const BwdArgs &a, const BwdPlan &p, hipStream_t s) {
  constexpr int CH = kChunk<T, R>;
  if (a.cols < CH) launch_cols<T, R, false, true, true, kOnce, 1, 8>(a, p, s);
  else if (p.lanes == 8) launch_cols<T, R, false, true, true, kOnce, CH, 8>(a, p, s);
  else if (p.lanes == 16) launch_cols<T, R, false, true, true, kOnce, CH, 16>(a, p, s);
  else if (p.lanes == 32) launch_cols<T, R, false, true, true, kOnce, CH, 32>(a, p, s);
  else launch_cols<T, R, false, true, true, kOnce, CH, 64>(a, p, s);
}

template <class T, class R, bool kX, bool kBias>
static void norm_bwd_of(const BwdArgs &a, const BwdPlan &p, hipStream_t s) {
  if (p.strips) {  // wide rows
    hipLaunchKernelGGL((k_row_stats<T, R>), dim3(row_grid(a.rows, 1u << 16)), dim3(1024), 0, s, a);
    if (a.once) launch_cols<T, R, true, kX, kBias, true, kChunk<T, R>, 64>(a, p, s);
    else launch_cols<T, R, true, kX, kBias, false, kChunk<T, R>, 64>(a, p, s);
  } else if (a.once) {
    norm_bwd_as<T, R, kX, kBias, true>(a, p, s);
  } else {
    norm_bwd_as<T, R, kX, kBias, false>(a, p, s);
  }
}

template <class TI, class TO, bool kDivide, class TP, bool kOnce>
static void drop_add_as(const AddArgs &a, int chunk, hipStream_t s) {
  const dim3 g((a.chunks + 255) / 256);
  if (chunk == 1) hipLaunchKernelGGL((k_drop_add<TI, TO, kDivide, kOnce, false, 1, TP>), g, dim3(256), 0, s, a);
  else if (a.flat) hipLaunchKernelGGL((k_drop_add<TI, TO, kDivide, kOnce, true, kChunk<TI, TO>, TP>), g, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_drop_add<TI, TO, kDivide, kOnce, false, kChunk<TI, TO>, TP>), g, dim3(256), 0, s, a);
}

template <class TI, class TO, class TP>
static void drop_add_of(const AddArgs &a, int chunk, hipStream_t s) {
  constexpr bool kDivide = std::is_same<TP, float>::value;
  if (a.once) drop_add_as<TI, TO, kDivide, TP, true>(a, chunk, s);
  else drop_add_as<TI, TO, kDivide, TP, false>(a, chunk, s);
}

template <class T, class R>
struct RowKernels {
  static void norm_fwd(const FwdArgs &a, hipStream_t s) {
    if (a.x) {
      if (a.once) norm_fwd_of<T, R, true, true>(a, s);
      else norm_fwd_of<T, R, true, false>(a, s);
    } else {
      if (a.once) norm_fwd_of<T, R, false, true>(a, s);
      else norm_fwd_of<T, R, false, false>(a, s);
    }
  }
  static void norm_bwd(const BwdArgs &a, const BwdPlan &p, bool bias, hipStream_t s) {
    if (!a.dx) norm_bwd_of<T, R, false, false>(a, p, s);
    else if (!bias) norm_bwd_of<T, R, true, false>(a, p, s);
    else norm_bwd_of<T, R, true, true>(a, p, s);
  }
  static void add_bwd_sums(const BwdArgs &a, const BwdPlan &p, hipStream_t s) {
    if (a.once) add_bwd_as<T, R, true>(a, p, s);
    else add_bwd_as<T, R, false>(a, p, s);
  }
  static void add_fwd(const AddArgs &a, int chunk, hipStream_t s) { drop_add_of<T, R, T>(a, chunk, s); }
  static void add_bwd(const AddArgs &a, int chunk, hipStream_t s) { drop_add_of<R, T, T>(a, chunk, s); }
  static RowTable table() { return {kChunk<T, R>, norm_fwd, norm_bwd, add_bwd_sums, add_fwd, add_bwd}; }
};

}  // namespace tk
