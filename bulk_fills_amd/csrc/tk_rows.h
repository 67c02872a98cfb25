// tk_rows.h -- kernels of the row operators (dropout-add, layer norm, both fused) for one
// pair of types: T of the activations, R of the residual stream.  Instantiated by
// tk_rows_f32.hip, tk_rows_f16.hip and tk_rows_bf16.hip; the C entry points are in
// tk_rows.hip.
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

// Data that is read once, past the caches.
template <int CH, class T>
__device__ __forceinline__ Chunk<T, CH> load_once(const T *p) {
  return __builtin_nontemporal_load((const Chunk<T, CH> *)p);
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

// Holds a chunk in its loaded form up to here: what is unpacked from it afterwards is unpacked
// again, so that two uses of a chunk on both sides of a row's sum do not keep its floats alive.
template <class C>
__device__ __forceinline__ void stay_packed(C &c) {
  if constexpr (sizeof(C) >= 8) {
    typedef uint32_t words __attribute__((ext_vector_type(sizeof(C) / 4)));
    words w = __builtin_bit_cast(words, c);
    __asm__ volatile("" : "+v"(w));
    c = __builtin_bit_cast(C, w);
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
// Kept values over 1 - p: the IEEE quotient for float, and a product with the reciprocal for
// the 16-bit types, whose 2^-23 relative error is far below their own rounding (2^-11, 2^-8).
template <bool kDivide, int CH>
__device__ __forceinline__ void drop_chunk(const Drop &d, uint32_t c, float *v) {
#pragma unroll
  for (int e = 0; e < CH; ++e) {
    const bool keep = (tk_word(d.hk, c + e) & 0x7FFFFFu) >= d.threshold;
    v[e] = keep ? (kDivide ? __fdiv_rn(v[e], d.q) : v[e] * d.rq) : 0.0f;
  }
}

// ---- sums over a row's lanes -----------------------------------------------------------
template <int kCtrl>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), kCtrl, 0xF, 0xF, true));
}

// The sum over each group of kLanes lanes (a power of two), the same bits in all of them:
// pairs, quads, then mirrored halves within 16 lanes, then the row swaps of gfx950.
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float x) {
  if (kLanes >= 2) x += dpp<0xB1>(x);    // quad_perm 1,0,3,2
  if (kLanes >= 4) x += dpp<0x4E>(x);    // quad_perm 2,3,0,1
  if (kLanes >= 8) x += dpp<0x141>(x);   // row_half_mirror
  if (kLanes >= 16) x += dpp<0x140>(x);  // row_mirror
  if (kLanes == 64) {
    const uint32_t u = __float_as_uint(x);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const uint32_t w = __float_as_uint(x);
    const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    x = __uint_as_float(b[0]) + __uint_as_float(b[1]);
  }
  return x;
}

// kN sums over the kTpr threads of a row.  Rows of up to a wave stay in registers; wider ones
// go through `slot` (kN floats a wave of the work-group), which must not be written again before
// another barrier has passed: every lane reads one wave's sums and the lanes add them up.
template <int kTpr, int kN>
__device__ __forceinline__ void row_sums(float (&x)[kN], float (*slot)[kN]) {
#pragma unroll
  for (int k = 0; k < kN; ++k) x[k] = lanes_sum<(kTpr < 64 ? kTpr : 64)>(x[k]);
  if constexpr (kTpr > 64) {
    constexpr uint32_t kWaves = kTpr / 64;
    const uint32_t wave = threadIdx.x >> 6, from = threadIdx.x / kTpr * kWaves + threadIdx.x % kWaves;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < kN; ++k) slot[wave][k] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kN; ++k) x[k] = lanes_sum<kWaves>(slot[from][k]);
  }
}

// The row group of a thread: on the scalar unit where a wave has one row, and with it the
// addresses of its rows.
template <int kTpr>
__device__ __forceinline__ uint32_t row_group() {
  const uint32_t g = threadIdx.x / kTpr;
  return kTpr >= 64 ? (uint32_t)__builtin_amdgcn_readfirstlane(g) : g;
}

// ---- forward ---------------------------------------------------------------------------
// A chunk of a row's inputs as loaded.
template <class T, class R, bool kX, int CH>
struct FwdIn {
  Chunk<T, CH> x;
  Chunk<R, CH> r;
  __device__ __forceinline__ void load(const FwdArgs &a, uint64_t row, uint32_t c) {
    const uint32_t at = chunk_at<CH>(c, a.cols);
    if constexpr (kX) x = load_once<CH>((const T *)a.x + row * a.ldx + at);
    if (!kX || a.residual) r = load_once<CH>((const R *)a.residual + row * a.ldr + at);
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

template <class T, class R, int CH>
__device__ __forceinline__ void norm_out(const FwdArgs &a, uint64_t row, uint32_t c, float mean, float rstd,
                                         const float *gamma, const float *beta, const float *v) {
  const int nv = (int)(a.cols - c);
  if (nv <= 0) return;
  if (a.sum) store_chunk<CH>((R *)a.sum + row * a.lds + c, nv, v);
  float y[CH];
#pragma unroll
  for (int e = 0; e < CH; ++e) y[e] = __builtin_fmaf((v[e] - mean) * rstd, gamma[e], beta[e]);
  store_chunk<CH>((T *)a.y + row * a.ldy + c, nv, y);
}

__device__ __forceinline__ float rstd_of(float m2, uint32_t cols, float eps) {
  return 1.0f / sqrtf(m2 / (float)cols + eps);
}

// The row stays in registers between the two sums (the mean, then the squared distances from
// it: no cancellation) and the output: one read and one write of the data.  A work-group takes
// every gridDim.x-th set of rows, keeps the parameters in registers, and loads its next rows
// before it works on the present ones.
template <class T, class R, bool kX, int CH, int kTpr, int V, int kBlk>
__global__ __launch_bounds__(kBlk) void k_norm_fwd(FwdArgs a) {
  constexpr int kRows = kBlk / kTpr;
  __shared__ float slot[2][kBlk / 64][1];
  const uint32_t t = threadIdx.x % kTpr;
  const uint64_t step = (uint64_t)gridDim.x * kRows;
  uint64_t row = (uint64_t)blockIdx.x * kRows + row_group<kTpr>();
  float bias[V][CH], gamma[V][CH], beta[V][CH];
  FwdIn<T, R, kX, CH> next[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t c = (j * kTpr + t) * CH;
    if (row < a.rows) next[j].load(a, row, c);
    if (kX) load_param<CH, T>(a.bias, a.params_f32, c, a.cols, 0.0f, bias[j]);
    load_param<CH, T>(a.gamma, a.params_f32, c, a.cols, 1.0f, gamma[j]);
    load_param<CH, T>(a.beta, a.params_f32, c, a.cols, 0.0f, beta[j]);
  }
  // every wave of a work-group runs the same rounds: the sums have barriers
  for (uint64_t base = (uint64_t)blockIdx.x * kRows; base < a.rows; base += step, row += step) {
    float v[V][CH], s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      next[j].value(a, row, (j * kTpr + t) * CH, bias[j], v[j]);
#pragma unroll
      for (int e = 0; e < CH; ++e) s[0] += v[j][e];
    }
    if (row + step < a.rows)
#pragma unroll
      for (int j = 0; j < V; ++j) next[j].load(a, row + step, (j * kTpr + t) * CH);
    row_sums<kTpr>(s, slot[0]);
    const float mean = s[0] / (float)a.cols;
    float m2[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int nv = (int)(a.cols - (j * kTpr + t) * CH);
      if (nv < CH)  // past the end: no distance from the mean
#pragma unroll
        for (int e = 0; e < CH; ++e) v[j][e] = e < nv ? v[j][e] : mean;
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        const float d = v[j][e] - mean;
        m2[0] = __builtin_fmaf(d, d, m2[0]);
      }
    }
    row_sums<kTpr>(m2, slot[1]);
    const float rstd = rstd_of(m2[0], a.cols, a.eps);
    if (row < a.rows) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        norm_out<T, R, CH>(a, row, (j * kTpr + t) * CH, mean, rstd, gamma[j], beta[j], v[j]);
      if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
    }
  }
}

// Rows too wide for the registers of one work-group: the same sums over three passes, the
// inputs read again in each (a row of some hundred KB stays in the caches).  Nothing is
// written before the third pass, and there each element's inputs are read by the thread
// that writes it, so outputs in place of inputs are fine.
template <class T, class R, bool kX>
__global__ __launch_bounds__(1024) void k_norm_fwd_wide(FwdArgs a) {
  constexpr int CH = kChunk<T, R>, kTpr = 1024;
  __shared__ float slot[2][kTpr / 64][1];
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const auto chunk = [&](uint32_t c, float *v) {
      FwdIn<T, R, kX, CH> in;
      float bias[CH];
      in.load(a, row, c);
      if (kX) load_param<CH, T>(a.bias, a.params_f32, c, a.cols, 0.0f, bias);
      in.value(a, row, c, bias, v);
    };
    float v[CH], s[1] = {0.0f};
    for (uint32_t c = threadIdx.x * CH; c < a.cols; c += kTpr * CH) {
      chunk(c, v);
      const int nv = (int)(a.cols - c);
#pragma unroll
      for (int e = 0; e < CH; ++e) s[0] += e < nv ? v[e] : 0.0f;
    }
    row_sums<kTpr>(s, slot[0]);
    const float mean = s[0] / (float)a.cols;
    float m2[1] = {0.0f};
    for (uint32_t c = threadIdx.x * CH; c < a.cols; c += kTpr * CH) {
      chunk(c, v);
      const int nv = (int)(a.cols - c);
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        const float d = e < nv ? v[e] - mean : 0.0f;
        m2[0] = __builtin_fmaf(d, d, m2[0]);
      }
    }
    row_sums<kTpr>(m2, slot[1]);
    const float rstd = rstd_of(m2[0], a.cols, a.eps);
    for (uint32_t c = threadIdx.x * CH; c < a.cols; c += kTpr * CH) {
      float gamma[CH], beta[CH];
      chunk(c, v);
      load_param<CH, T>(a.gamma, a.params_f32, c, a.cols, 1.0f, gamma);
      load_param<CH, T>(a.beta, a.params_f32, c, a.cols, 0.0f, beta);
      norm_out<T, R, CH>(a, row, c, mean, rstd, gamma, beta, v);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// ---- backward --------------------------------------------------------------------------
// Layer norm's gradient for one element: rstd (g - mean(g) - h mean(g h)).
__device__ __forceinline__ float norm_grad(float g, float h, float rstd, float mg, float mgh) {
  return rstd * __builtin_fmaf(-h, mgh, g - mg);
}

// A chunk of a row's inputs as loaded.  dy is of type D: T, or R for dropout-add's gradient.
template <class T, class R, class D, bool kNorm, int CH>
struct BwdIn {
  Chunk<D, CH> dy;
  Chunk<R, CH> sum, dsum;
  __device__ __forceinline__ void load(const BwdArgs &a, uint64_t row, uint32_t c) {
    const uint32_t at = chunk_at<CH>(c, a.cols);
    dy = load_once<CH>((const D *)a.dy + row * a.lddy + at);
    if (kNorm) sum = load_once<CH>((const R *)a.sum + row * a.lds + at);
    if (a.dsum) dsum = load_once<CH>((const R *)a.dsum + row * a.ldds + at);
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

// Rows in registers, as forward: as loaded, between the sums and the output.  A work-group
// takes every gridDim.x-th set of rows and keeps the column sums of its own rows in registers;
// at the end its groups' sums are added up through LDS and written to the workspace, one line
// of partial sums per work-group, which k_finish adds up in order.
template <class T, class R, bool kX, bool kBias, int CH, int kTpr, int V, int kBlk>
__global__ __launch_bounds__(kBlk) void k_norm_bwd(BwdArgs a) {
  constexpr int kRows = kBlk / kTpr, kSums = kBias ? 3 : 2;
  __shared__ float slot[2][kBlk / 64][2];
  const uint32_t t = threadIdx.x % kTpr, group = row_group<kTpr>();
  const uint64_t step = (uint64_t)gridDim.x * kRows;
  uint64_t row = (uint64_t)blockIdx.x * kRows + group;
  const float inv = 1.0f / (float)a.cols;
  float acc[kSums][V][CH], gamma[V][CH], mean = 0.0f, rstd = 0.0f;
  BwdIn<T, R, T, true, CH> next[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t c = (j * kTpr + t) * CH;
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
  for (uint64_t base = (uint64_t)blockIdx.x * kRows; base < a.rows; base += step, row += step, par ^= 1) {
    const bool here = row < a.rows;
    const float m = mean, rs = rstd;
    BwdIn<T, R, T, true, CH> in[V];
#pragma unroll
    for (int j = 0; j < V; ++j) in[j] = next[j];
    if (row + step < a.rows) {
#pragma unroll
      for (int j = 0; j < V; ++j) next[j].load(a, row + step, (j * kTpr + t) * CH);
      mean = a.mean[row + step];
      rstd = a.rstd[row + step];
    }
    float s[2] = {0.0f, 0.0f};
    if (here) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int nv = (int)(a.cols - (j * kTpr + t) * CH);
        float g[CH], h[CH];
        unpack<CH, T>(in[j].dy, nv, g);
        in[j].normed(nv, m, rs, h);
#pragma unroll
        for (int e = 0; e < CH; ++e) {
          acc[0][j][e] = __builtin_fmaf(g[e], h[e], acc[0][j][e]);
          acc[1][j][e] += g[e];
          const float w = g[e] * gamma[j][e];
          s[0] += w;
          s[1] = __builtin_fmaf(w, h[e], s[1]);
        }
      }
    }
    row_sums<kTpr>(s, slot[par]);
    if (here) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t c = (j * kTpr + t) * CH;
        const int nv = (int)(a.cols - c);
        float g[CH], h[CH];
        stay_packed(in[j].dy);
        stay_packed(in[j].sum);
        unpack<CH, T>(in[j].dy, nv, g);
        in[j].normed(nv, m, rs, h);
#pragma unroll
        for (int e = 0; e < CH; ++e) g[e] = norm_grad(g[e] * gamma[j][e], h[e], rs, s[0] * inv, s[1] * inv);
        in[j].template out<kX>(a, row, c, g);
        if constexpr (kBias) {
#pragma unroll
          for (int e = 0; e < CH; ++e) acc[2][j][e] += g[e];
        }
      }
    }
  }
  if (!a.partial) return;
  constexpr int kCols = kTpr * V * CH;
  __shared__ float tile[kRows > 1 ? kRows : 1][kRows > 1 ? kCols : 1];
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
    float *line = a.partial + ((uint64_t)k * gridDim.x + blockIdx.x) * a.cols;
    if constexpr (kRows > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < CH; ++e) tile[group][(j * kTpr + t) * CH + e] = acc[k][j][e];
      __syncthreads();
      for (uint32_t c = threadIdx.x; c < kCols && c < a.cols; c += kBlk) {
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) s += tile[r][c];
        line[c] = s;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t c = (j * kTpr + t) * CH;
        const int nv = (int)(a.cols - c);
#pragma unroll
        for (int e = 0; e < CH; ++e)
          if (e < nv) line[c + e] = acc[k][j][e];
      }
    }
  }
}

// Rows wider than k_norm_bwd's registers hold with their column sums: first mean(g) and
// mean(g h) of every row, then k_cols_bwd over columns.
template <class T, class R>
__global__ __launch_bounds__(1024) void k_row_stats(BwdArgs a) {
  constexpr int CH = kChunk<T, R>, kTpr = 1024;
  __shared__ float slot[2][kTpr / 64][2];
  int par = 0;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, par ^= 1) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s[2] = {0.0f, 0.0f};
    for (uint32_t c = threadIdx.x * CH; c < a.cols; c += kTpr * CH) {
      const int nv = (int)(a.cols - c);
      const uint32_t at = chunk_at<CH>(c, a.cols);
      float g[CH], h[CH], w[CH];
      // read again by k_cols_bwd: kept in the caches
      unpack<CH, T>(*(const Chunk<T, CH> *)((const T *)a.dy + row * a.lddy + at), nv, g);
      unpack<CH, R>(*(const Chunk<R, CH> *)((const R *)a.sum + row * a.lds + at), nv, h);
      load_param<CH, T>(a.gamma, a.params_f32, c, a.cols, 1.0f, w);
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        const float x = g[e] * w[e];
        s[0] += x;
        s[1] = __builtin_fmaf(x, (h[e] - mean) * rstd, s[1]);
      }
    }
    row_sums<kTpr>(s, slot[par]);
    if (threadIdx.x == 0) {
      a.stats[2 * row] = s[0] / (float)a.cols;
      a.stats[2 * row + 1] = s[1] / (float)a.cols;
    }
  }
}

// A strip of 64 lanes' chunks by a range of rows, four waves taking every fourth row: each
// lane keeps the sums of its own columns.  kNorm: layer norm's gradient with the row's means
// from k_row_stats; else dy (of the residual stream's type) is the sum's gradient itself.
template <class T, class R, bool kNorm, bool kX, bool kBias, int CH>
__global__ __launch_bounds__(256) void k_cols_bwd(BwdArgs a) {
  constexpr int kSums = (kNorm ? 2 : 0) + (kBias ? 1 : 0);
  typedef typename std::conditional<kNorm, T, R>::type D;
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t c = (blockIdx.x * 64 + lane) * CH;
  const int nv = (int)(a.cols - c);
  const uint64_t r0 = (uint64_t)blockIdx.y * a.rows_per_block;
  const uint64_t r1 = r0 + a.rows_per_block < a.rows ? r0 + a.rows_per_block : a.rows;
  float acc[kSums ? kSums : 1][CH];
#pragma unroll
  for (int k = 0; k < kSums; ++k)
#pragma unroll
    for (int e = 0; e < CH; ++e) acc[k][e] = 0.0f;
  if (nv > 0) {
    float w[CH];
    if (kNorm) load_param<CH, T>(a.gamma, a.params_f32, c, a.cols, 1.0f, w);
#pragma unroll 2
    for (uint64_t row = r0 + wave; row < r1; row += 4) {
      BwdIn<T, R, D, kNorm, CH> in;
      in.load(a, row, c);
      float v[CH];
      unpack<CH, D>(in.dy, nv, v);
      if constexpr (kNorm) {
        const float rstd = a.rstd[row], mg = a.stats[2 * row], mgh = a.stats[2 * row + 1];
        float h[CH];
        in.normed(nv, a.mean[row], rstd, h);
#pragma unroll
        for (int e = 0; e < CH; ++e) {
          acc[0][e] = __builtin_fmaf(v[e], h[e], acc[0][e]);
          acc[1][e] += v[e];
          v[e] = norm_grad(v[e] * w[e], h[e], rstd, mg, mgh);
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
    if (!a.partial) return;
    __shared__ float tile[4][64 * CH];
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
      if (k) __syncthreads();
#pragma unroll
      for (int e = 0; e < CH; ++e) tile[wave][e * 64 + lane] = acc[k][e];
      __syncthreads();
      float *line = a.partial + ((uint64_t)k * gridDim.y + blockIdx.y) * a.cols;
      for (uint32_t i = threadIdx.x; i < 64 * CH; i += 256) {
        const uint32_t e = i % CH, l = i / CH, col = blockIdx.x * 64 * CH + i;
        if (col < a.cols)
          line[col] = (tile[0][e * 64 + l] + tile[1][e * 64 + l]) + (tile[2][e * 64 + l] + tile[3][e * 64 + l]);
      }
    }
  }
}

// ---- dropout-add, element by element ---------------------------------------------------
// Chunk n of the call lies in row n / chunks_per_row (a product with the rounded-up
// reciprocal: exact below 2^31 chunks, which a launch stays under).
template <class TI, class TO, bool kDivide, int CH, class TP>
__global__ __launch_bounds__(256) void k_drop_add(AddArgs a) {
  const uint32_t n = blockIdx.x * 256u + threadIdx.x;
  if (n >= a.chunks) return;
  const uint32_t r = a.div_shift < 0 ? n : __umulhi(n, a.div_mul) >> a.div_shift;
  const uint64_t c = (uint64_t)(n - r * a.chunks_per_row) * CH, row = a.row0 + r, at = chunk_at<CH>(c, a.cols64);
  const int nv = a.cols64 - c < CH ? (int)(a.cols64 - c) : CH;
  const Chunk<TI, CH> x = load_once<CH>((const TI *)a.x + row * a.ldx + at);
  Chunk<TO, CH> d;
  if (a.residual) d = load_once<CH>((const TO *)a.residual + row * a.ldr + at);
  float v[CH];
  if (a.bias) {
    float b[CH];
    load_param<CH, TP>(a.bias, a.params_f32, (uint32_t)c, (uint32_t)a.cols64, 0.0f, b);
    unpack<CH, TI>(x, nv, v);
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] += b[e];
  } else {
    unpack<CH, TI>(x, nv, v);
  }
  if (a.drop.on) drop_chunk<kDivide, CH>(a.drop, a.drop.start + (uint32_t)(row * a.cols64 + c), v);
  if (a.residual) {
    float u[CH];
    unpack<CH, TO>(d, nv, u);
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] += u[e];
  }
  store_chunk<CH>((TO *)a.y + row * a.ldy + c, nv, v);
}

// ---- launches --------------------------------------------------------------------------
// Work-groups over sets of rows; the kernels loop beyond (a launch holds fewer than 2^32 threads).
static inline uint32_t row_grid(uint64_t sets, uint32_t most) { return (uint32_t)(sets < most ? sets : most); }

#ifndef TK_FWD_GRID
#define TK_FWD_GRID 1024
#endif
template <class T, class R, bool kX, int CH, int kTpr, int V, int kBlk>
static void launch_fwd(const FwdArgs &a, hipStream_t s) {
  constexpr int kRows = kBlk / kTpr;
  hipLaunchKernelGGL((k_norm_fwd<T, R, kX, CH, kTpr, V, kBlk>), dim3(row_grid((a.rows + kRows - 1) / kRows, TK_FWD_GRID)),
                     dim3(kBlk), 0, s, a);
}

template <class T, class R, bool kX>
static void norm_fwd_of(const FwdArgs &a, hipStream_t s) {
  constexpr int CH = kChunk<T, R>, K = 8 / CH;
  if (a.cols < CH) launch_fwd<T, R, kX, 1, 16, 1, 256>(a, s);
  else if (a.cols <= 128) launch_fwd<T, R, kX, CH, 16, K, 256>(a, s);
  else if (a.cols <= 512) launch_fwd<T, R, kX, CH, 64, K, 256>(a, s);
  else if (a.cols <= 1024) launch_fwd<T, R, kX, CH, 64, 2 * K, 256>(a, s);
  else if (a.cols <= 2048) launch_fwd<T, R, kX, CH, 256, K, 256>(a, s);
  else if (a.cols <= 4096) launch_fwd<T, R, kX, CH, 512, K, 512>(a, s);
  else if (a.cols <= 8192) launch_fwd<T, R, kX, CH, 1024, K, 1024>(a, s);
  else if (a.cols <= 16384) launch_fwd<T, R, kX, CH, 1024, 2 * K, 1024>(a, s);
  else hipLaunchKernelGGL((k_norm_fwd_wide<T, R, kX>), dim3(row_grid(a.rows, 1u << 16)), dim3(1024), 0, s, a);
}

template <class T, class R, bool kX, bool kBias>
static void norm_bwd_of(const BwdArgs &a, const BwdPlan &p, hipStream_t s) {
  constexpr int CH = kChunk<T, R>, K = 8 / CH;
  const dim3 g((uint32_t)p.lines);
#define TK_BWD(CHUNK, TPR, V, BLK) \
  hipLaunchKernelGGL((k_norm_bwd<T, R, kX, kBias, CHUNK, TPR, V, BLK>), g, dim3(BLK), 0, s, a)
  if (a.cols < CH) TK_BWD(1, 16, 1, 256);
  else if (p.tpr == 16) TK_BWD(CH, 16, K, 512);
  else if (p.tpr == 64) TK_BWD(CH, 64, K, 512);
  else if (p.tpr == 128) TK_BWD(CH, 128, K, 512);
  else if (p.tpr == 256) TK_BWD(CH, 256, K, 512);
  else if (p.tpr == 512) TK_BWD(CH, 512, K, 512);
  else if (p.ept == 8) TK_BWD(CH, 1024, K, 1024);
  else TK_BWD(CH, 1024, 2 * K, 1024);
#undef TK_BWD
}

template <class T, class R, bool kNorm, bool kX, bool kBias>
static void cols_bwd_of(const BwdArgs &a, const BwdPlan &p, hipStream_t s) {
  const dim3 g((uint32_t)p.strips, (uint32_t)p.lines);
  if (!kNorm && a.cols < kChunk<T, R>)
    hipLaunchKernelGGL((k_cols_bwd<T, R, kNorm, kX, kBias, kNorm ? kChunk<T, R> : 1>), g, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_cols_bwd<T, R, kNorm, kX, kBias, kChunk<T, R>>), g, dim3(256), 0, s, a);
}

template <class TI, class TO, bool kDivide, class TP>
static void drop_add_of(const AddArgs &a, int chunk, hipStream_t s) {
  const dim3 g((a.chunks + 255) / 256);
  if (chunk == 1) hipLaunchKernelGGL((k_drop_add<TI, TO, kDivide, 1, TP>), g, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_drop_add<TI, TO, kDivide, kChunk<TI, TO>, TP>), g, dim3(256), 0, s, a);
}

template <class T, class R>
struct RowKernels {
  static void norm_fwd(const FwdArgs &a, hipStream_t s) {
    if (a.x) norm_fwd_of<T, R, true>(a, s);
    else norm_fwd_of<T, R, false>(a, s);
  }
  static void norm_bwd(const BwdArgs &a, const BwdPlan &p, bool bias, hipStream_t s) {
    if (p.tpr == 0) {  // wide rows
      hipLaunchKernelGGL((k_row_stats<T, R>), dim3(row_grid(a.rows, 1u << 16)), dim3(1024), 0, s, a);
      if (!a.dx) cols_bwd_of<T, R, true, false, false>(a, p, s);
      else if (!bias) cols_bwd_of<T, R, true, true, false>(a, p, s);
      else cols_bwd_of<T, R, true, true, true>(a, p, s);
      return;
    }
    if (!a.dx) norm_bwd_of<T, R, false, false>(a, p, s);
    else if (!bias) norm_bwd_of<T, R, true, false>(a, p, s);
    else norm_bwd_of<T, R, true, true>(a, p, s);
  }
  static void add_bwd_sums(const BwdArgs &a, const BwdPlan &p, hipStream_t s) {
    cols_bwd_of<T, R, false, true, true>(a, p, s);
  }
  static void add_fwd(const AddArgs &a, int chunk, hipStream_t s) {
    drop_add_of<T, R, std::is_same<T, float>::value, T>(a, chunk, s);
  }
  static void add_bwd(const AddArgs &a, int chunk, hipStream_t s) {
    drop_add_of<R, T, std::is_same<T, float>::value, T>(a, chunk, s);
  }
  static RowTable table() { return {kChunk<T, R>, norm_fwd, norm_bwd, add_bwd_sums, add_fwd, add_bwd}; }
};

}  // namespace tk
