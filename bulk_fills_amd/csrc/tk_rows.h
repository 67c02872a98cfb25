// tk_rows.h -- kernels of the row operators (dropout-add, layer norm, both fused) for one
// pair of types: T of the activations, R of the residual stream.  Instantiated by
// tk_rows_f32.hip, tk_rows_f16.hip and tk_rows_bf16.hip; the C entry points are in
// tk_rows.hip.
//
// A lane handles chunks of kChunk consecutive elements of a row: 16 bytes of the wider of
// the two types.  Addresses need only element alignment (gfx950 takes vector loads and
// stores at any), so odd widths and row pitches run the same code; the one chunk of a row
// that reaches past its end goes element by element.
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
// The first nv elements of the CH at p, as floats (the rest 0).
template <int CH, class T>
__device__ __forceinline__ void load_chunk(const T *p, int nv, float *v) {
  typedef T vec __attribute__((ext_vector_type(CH), aligned(sizeof(T))));
  if (nv >= CH) {
    const vec t = *(const vec *)p;
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] = (float)t[e];
  } else {
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] = e < nv ? (float)p[e] : 0.0f;
  }
}

template <int CH, class T>
__device__ __forceinline__ void store_chunk(T *p, int nv, const float *v) {
  typedef T vec __attribute__((ext_vector_type(CH), aligned(sizeof(T))));
  if (nv >= CH) {
    vec t;
#pragma unroll
    for (int e = 0; e < CH; ++e) t[e] = (T)v[e];  // round to nearest even
    *(vec *)p = t;
  } else {
#pragma unroll
    for (int e = 0; e < CH; ++e)
      if (e < nv) p[e] = (T)v[e];
  }
}

// A parameter vector's chunk at column c: float or T elements, `other` where there is none.
template <int CH, class T>
__device__ __forceinline__ void load_param(const void *p, bool f32, uint32_t c, int nv, float other, float *v) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] = other;
  } else if (f32) {
    load_chunk<CH>((const float *)p + c, nv, v);
  } else {
    load_chunk<CH>((const T *)p + c, nv, v);
  }
}

// ---- dropout ---------------------------------------------------------------------------
// Kept values over 1 - p: the IEEE quotient for float, and a product with the reciprocal for
// the 16-bit types, whose 2^-24 relative error is far below their own rounding (2^-12, 2^-9).
template <bool kDivide>
__device__ __forceinline__ float drop_one(const Drop &d, uint32_t c, float v) {
  const bool keep = (tk_word(d.hk, c) & 0x7FFFFFu) >= d.threshold;
  return keep ? (kDivide ? __fdiv_rn(v, d.q) : v * d.rq) : 0.0f;
}

template <bool kDivide, int CH>
__device__ __forceinline__ void drop_chunk(const Drop &d, uint32_t c, float *v) {
#pragma unroll
  for (int e = 0; e < CH; ++e) v[e] = drop_one<kDivide>(d, c + e, v[e]);
}

// ---- sums over a row's lanes -----------------------------------------------------------
template <int kCtrl>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), kCtrl, 0xF, 0xF, true));
}

// The sum over each group of kLanes (16 or 64) lanes, the same bits in all of them: pairs,
// quads, then mirrored halves within 16 lanes, then the row swaps of gfx950.
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float x) {
  x += dpp<0xB1>(x);   // quad_perm 1,0,3,2
  x += dpp<0x4E>(x);   // quad_perm 2,3,0,1
  x += dpp<0x141>(x);  // row_half_mirror
  x += dpp<0x140>(x);  // row_mirror
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

// Two sums over the kTpr threads of a row.  Rows of up to a wave stay in registers; wider
// ones go through `slot` (2 floats a wave), which must not be written again before another
// barrier has passed.
template <int kTpr>
__device__ __forceinline__ void row_sums(float &x, float &y, float (*slot)[2]) {
  x = lanes_sum<(kTpr < 64 ? kTpr : 64)>(x);
  y = lanes_sum<(kTpr < 64 ? kTpr : 64)>(y);
  if constexpr (kTpr > 64) {
    const uint32_t wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      slot[wave][0] = x;
      slot[wave][1] = y;
    }
    __syncthreads();
    x = y = 0.0f;
#pragma unroll
    for (int w = 0; w < kTpr / 64; ++w) {
      x += slot[w][0];
      y += slot[w][1];
    }
  }
}

template <int kTpr>
__device__ __forceinline__ float row_sum(float x, float (*slot)[2]) {
  x = lanes_sum<(kTpr < 64 ? kTpr : 64)>(x);
  if constexpr (kTpr > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6][0] = x;
    __syncthreads();
    x = 0.0f;
#pragma unroll
    for (int w = 0; w < kTpr / 64; ++w) x += slot[w][0];
  }
  return x;
}

// ---- forward ---------------------------------------------------------------------------
// One chunk of the norm's input: residual + drop(x + bias).
template <class T, class R, bool kX, int CH>
__device__ __forceinline__ void input_chunk(const FwdArgs &a, uint64_t row, uint32_t c, int nv, float *v) {
  if constexpr (kX) {
    load_chunk<CH>((const T *)a.x + row * a.ldx + c, nv, v);
    if (a.bias) {
      float b[CH];
      load_param<CH, T>(a.bias, a.params_f32, c, nv, 0.0f, b);
#pragma unroll
      for (int e = 0; e < CH; ++e) v[e] += b[e];
    }
    if (a.drop.on) drop_chunk<std::is_same<T, float>::value, CH>(a.drop, a.drop.start + (uint32_t)(row * a.cols) + c, v);
    if (a.residual) {
      float r[CH];
      load_chunk<CH>((const R *)a.residual + row * a.ldr + c, nv, r);
#pragma unroll
      for (int e = 0; e < CH; ++e) v[e] += r[e];
    }
  } else {
    load_chunk<CH>((const R *)a.residual + row * a.ldr + c, nv, v);
  }
}

template <class T, class R, int CH>
__device__ __forceinline__ void output_chunk(const FwdArgs &a, uint64_t row, uint32_t c, int nv, float mean, float rstd,
                                             const float *v) {
  if (a.sum) store_chunk<CH>((R *)a.sum + row * a.lds + c, nv, v);
  float g[CH], b[CH], y[CH];
  load_param<CH, T>(a.gamma, a.params_f32, c, nv, 1.0f, g);
  load_param<CH, T>(a.beta, a.params_f32, c, nv, 0.0f, b);
#pragma unroll
  for (int e = 0; e < CH; ++e) y[e] = __builtin_fmaf((v[e] - mean) * rstd, g[e], b[e]);
  store_chunk<CH>((T *)a.y + row * a.ldy + c, nv, y);
}

__device__ __forceinline__ float rstd_of(float m2, uint32_t cols, float eps) {
  return 1.0f / sqrtf(m2 / (float)cols + eps);
}

// The row stays in registers between the two sums (the mean, then the squared distances
// from it: no cancellation) and the output: one read and one write of the data.
template <class T, class R, bool kX, int kTpr, int kEpt>
__global__ __launch_bounds__(kTpr < 256 ? 256 : kTpr) void k_norm_fwd(FwdArgs a) {
  constexpr int CH = kChunk<T, R>, V = kEpt / CH, kRows = kTpr < 256 ? 256 / kTpr : 1;
  __shared__ float slot[2][kTpr > 64 ? kTpr / 64 : 1][2];
  const uint32_t t = threadIdx.x % kTpr;
  for (uint64_t row = (uint64_t)blockIdx.x * kRows + threadIdx.x / kTpr; row < a.rows; row += (uint64_t)gridDim.x * kRows) {
  float v[V][CH], s = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t c = (j * kTpr + t) * CH;
    const int nv = (int)(a.cols - c);
    if (nv > 0) {
      input_chunk<T, R, kX, CH>(a, row, c, nv, v[j]);
    }
    if (nv < CH) {
#pragma unroll
      for (int e = 0; e < CH; ++e) v[j][e] = e < nv ? v[j][e] : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < CH; ++e) s += v[j][e];
  }
  const float mean = row_sum<kTpr>(s, slot[0]) / (float)a.cols;
  float m2 = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int nv = (int)(a.cols - (j * kTpr + t) * CH);
    if (nv < CH) {  // past the end: no distance from the mean
#pragma unroll
      for (int e = 0; e < CH; ++e) v[j][e] = e < nv ? v[j][e] : mean;
    }
#pragma unroll
    for (int e = 0; e < CH; ++e) {
      const float d = v[j][e] - mean;
      m2 = __builtin_fmaf(d, d, m2);
    }
  }
  m2 = row_sum<kTpr>(m2, slot[1]);
  const float rstd = rstd_of(m2, a.cols, a.eps);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t c = (j * kTpr + t) * CH;
    const int nv = (int)(a.cols - c);
    if (nv > 0) output_chunk<T, R, CH>(a, row, c, nv, mean, rstd, v[j]);
  }
  if (t == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
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
  __shared__ float slot[2][kTpr / 64][2];
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
  float v[CH], s = 0.0f;
  for (uint32_t c = threadIdx.x * CH; c < a.cols; c += kTpr * CH) {
    const int nv = (int)(a.cols - c);
    input_chunk<T, R, kX, CH>(a, row, c, nv, v);
#pragma unroll
    for (int e = 0; e < CH; ++e) s += e < nv ? v[e] : 0.0f;
  }
  const float mean = row_sum<kTpr>(s, slot[0]) / (float)a.cols;
  float m2 = 0.0f;
  for (uint32_t c = threadIdx.x * CH; c < a.cols; c += kTpr * CH) {
    const int nv = (int)(a.cols - c);
    input_chunk<T, R, kX, CH>(a, row, c, nv, v);
#pragma unroll
    for (int e = 0; e < CH; ++e) {
      const float d = e < nv ? v[e] - mean : 0.0f;
      m2 = __builtin_fmaf(d, d, m2);
    }
  }
  m2 = row_sum<kTpr>(m2, slot[1]);
  const float rstd = rstd_of(m2, a.cols, a.eps);
  for (uint32_t c = threadIdx.x * CH; c < a.cols; c += kTpr * CH) {
    const int nv = (int)(a.cols - c);
    input_chunk<T, R, kX, CH>(a, row, c, nv, v);
    output_chunk<T, R, CH>(a, row, c, nv, mean, rstd, v);
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

// Outputs of one chunk: dresidual = v + dsum and dx = drop(dresidual), returned in v.
template <class T, class R, bool kX, int CH>
__device__ __forceinline__ void grad_chunk(const BwdArgs &a, uint64_t row, uint32_t c, int nv, float *v) {
  if (a.dsum) {
    float d[CH];
    load_chunk<CH>((const R *)a.dsum + row * a.ldds + c, nv, d);
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] += d[e];
  }
  if (a.dresidual) store_chunk<CH>((R *)a.dresidual + row * a.lddr + c, nv, v);
  if constexpr (kX) {
    if (a.drop.on) drop_chunk<std::is_same<T, float>::value, CH>(a.drop, a.drop.start + (uint32_t)(row * a.cols) + c, v);
    store_chunk<CH>((T *)a.dx + row * a.lddx + c, nv, v);
  }
}

// Rows in registers, as forward.  A work-group takes every gridDim.x-th set of rows and keeps
// the column sums of its own rows in registers; at the end it writes them to the workspace,
// one line of partial sums per work-group, which k_finish adds up in order.
template <class T, class R, bool kX, bool kBias, int kTpr, int kEpt>
__global__ __launch_bounds__(kTpr < 256 ? 256 : kTpr) void k_norm_bwd(BwdArgs a) {
  constexpr int CH = kChunk<T, R>, V = kEpt / CH, kRows = kTpr < 256 ? 256 / kTpr : 1;
  constexpr int kBlk = kTpr * kRows, kSums = kBias ? 3 : 2;
  __shared__ float slot[2][kTpr > 64 ? kTpr / 64 : 1][2];
  const uint32_t t = threadIdx.x % kTpr, group = threadIdx.x / kTpr;
  float acc[kSums][V][CH];
#pragma unroll
  for (int k = 0; k < kSums; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < CH; ++e) acc[k][j][e] = 0.0f;
  const float inv = 1.0f / (float)a.cols;
  int par = 0;  // the slot in use: one barrier a row keeps the other one safe to write
  for (uint64_t row = (uint64_t)blockIdx.x * kRows + group; row < a.rows; row += (uint64_t)gridDim.x * kRows) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    float g[V][CH], h[V][CH], sg = 0.0f, sgh = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t c = (j * kTpr + t) * CH;
      const int nv = (int)(a.cols - c);
      float w[CH];
      if (nv > 0) {
        load_chunk<CH>((const T *)a.dy + row * a.lddy + c, nv, g[j]);
        load_chunk<CH>((const R *)a.sum + row * a.lds + c, nv, h[j]);
        load_param<CH, T>(a.gamma, a.params_f32, c, nv, 1.0f, w);
      }
      if (nv < CH) {
#pragma unroll
        for (int e = 0; e < CH; ++e) {
          g[j][e] = e < nv ? g[j][e] : 0.0f;
          h[j][e] = e < nv ? h[j][e] : mean;
          w[e] = e < nv ? w[e] : 0.0f;
        }
      }
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        h[j][e] = (h[j][e] - mean) * rstd;
        acc[0][j][e] = __builtin_fmaf(g[j][e], h[j][e], acc[0][j][e]);
        acc[1][j][e] += g[j][e];
        g[j][e] *= w[e];
        sg += g[j][e];
        sgh = __builtin_fmaf(g[j][e], h[j][e], sgh);
      }
    }
    row_sums<kTpr>(sg, sgh, slot[par]);
    par ^= 1;
    sg *= inv;
    sgh *= inv;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t c = (j * kTpr + t) * CH;
      const int nv = (int)(a.cols - c);
      if (nv > 0) {
        float v[CH];
#pragma unroll
        for (int e = 0; e < CH; ++e) v[e] = norm_grad(g[j][e], h[j][e], rstd, sg, sgh);
        grad_chunk<T, R, kX, CH>(a, row, c, nv, v);
        if constexpr (kBias) {
#pragma unroll
          for (int e = 0; e < CH; ++e) acc[2][j][e] += v[e];
        }
      }
    }
  }
  if (!a.partial) return;
  // the groups of a work-group hold the same columns: added up through LDS, in order
  __shared__ float tile[kRows > 1 ? kBlk * kEpt : 1];
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
    float *line = a.partial + ((uint64_t)k * gridDim.x + blockIdx.x) * a.cols;
    if constexpr (kRows > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < CH; ++e) tile[(group * kEpt * kTpr) + (j * kTpr + t) * CH + e] = acc[k][j][e];
      __syncthreads();
      for (uint32_t c = threadIdx.x; c < kTpr * kEpt && c < a.cols; c += kBlk) {
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) s += tile[r * kEpt * kTpr + c];
        line[c] = s;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t c = (j * kTpr + t) * CH;
        const int nv = (int)(a.cols - c);
        if (nv > 0) store_chunk<CH>(line + c, nv, acc[k][j]);
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
  float sg = 0.0f, sgh = 0.0f;
  for (uint32_t c = threadIdx.x * CH; c < a.cols; c += kTpr * CH) {
    const int nv = (int)(a.cols - c);
    float g[CH], h[CH], w[CH];
    load_chunk<CH>((const T *)a.dy + row * a.lddy + c, nv, g);
    load_chunk<CH>((const R *)a.sum + row * a.lds + c, nv, h);
    load_param<CH, T>(a.gamma, a.params_f32, c, nv, 1.0f, w);
#pragma unroll
    for (int e = 0; e < CH; ++e) {
      const float x = e < nv ? g[e] * w[e] : 0.0f;
      sg += x;
      sgh = __builtin_fmaf(x, e < nv ? (h[e] - mean) * rstd : 0.0f, sgh);
    }
  }
  row_sums<kTpr>(sg, sgh, slot[par]);
  if (threadIdx.x == 0) {
    a.stats[2 * row] = sg / (float)a.cols;
    a.stats[2 * row + 1] = sgh / (float)a.cols;
  }
  }
}

// A strip of 64 lanes' chunks by a range of rows, four waves taking every fourth row: each
// lane keeps the sums of its own columns.  kNorm: layer norm's gradient with the row's means
// from k_row_stats; else dy (of the residual stream's type) is the sum's gradient itself.
template <class T, class R, bool kNorm, bool kX, bool kBias>
__global__ __launch_bounds__(256) void k_cols_bwd(BwdArgs a) {
  constexpr int CH = kChunk<T, R>, kSums = (kNorm ? 2 : 0) + (kBias ? 1 : 0);
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
    if (kNorm) load_param<CH, T>(a.gamma, a.params_f32, c, nv, 1.0f, w);
    for (uint64_t row = r0 + wave; row < r1; row += 4) {
      float v[CH];
      if constexpr (kNorm) {
        const float mean = a.mean[row], rstd = a.rstd[row], mg = a.stats[2 * row], mgh = a.stats[2 * row + 1];
        float g[CH], h[CH];
        load_chunk<CH>((const T *)a.dy + row * a.lddy + c, nv, g);
        load_chunk<CH>((const R *)a.sum + row * a.lds + c, nv, h);
#pragma unroll
        for (int e = 0; e < CH; ++e) {
          h[e] = (h[e] - mean) * rstd;
          acc[0][e] = __builtin_fmaf(g[e], h[e], acc[0][e]);
          acc[1][e] += g[e];
          v[e] = norm_grad(g[e] * w[e], h[e], rstd, mg, mgh);
        }
      } else {
        load_chunk<CH>((const R *)a.dy + row * a.lddy + c, nv, v);
      }
      grad_chunk<T, R, kX, CH>(a, row, c, nv, v);
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
  const uint64_t c = (uint64_t)(n - r * a.chunks_per_row) * CH, row = a.row0 + r;
  const int nv = a.cols64 - c < CH ? (int)(a.cols64 - c) : CH;
  float v[CH];
  load_chunk<CH>((const TI *)a.x + row * a.ldx + c, nv, v);
  if (a.bias) {
    float b[CH];
    load_param<CH, TP>(a.bias, a.params_f32, (uint32_t)c, nv, 0.0f, b);
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] += b[e];
  }
  if (a.drop.on) drop_chunk<kDivide, CH>(a.drop, a.drop.start + (uint32_t)(row * a.cols64 + c), v);
  if (a.residual) {
    float d[CH];
    load_chunk<CH>((const TO *)a.residual + row * a.ldr + c, nv, d);
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] += d[e];
  }
  store_chunk<CH>((TO *)a.y + row * a.ldy + c, nv, v);
}

// ---- launches --------------------------------------------------------------------------
// Work-groups over sets of rows; the kernels loop beyond (a launch holds fewer than 2^32 threads).
static inline uint32_t row_grid(uint64_t sets) { return (uint32_t)(sets < (1u << 20) ? sets : (1u << 20)); }

template <class T, class R, bool kX, int kTpr, int kEpt>
static void launch_fwd(const FwdArgs &a, hipStream_t s) {
  constexpr int kRows = kTpr < 256 ? 256 / kTpr : 1;
  hipLaunchKernelGGL((k_norm_fwd<T, R, kX, kTpr, kEpt>), dim3(row_grid((a.rows + kRows - 1) / kRows)),
                     dim3(kTpr * kRows), 0, s, a);
}

template <class T, class R, bool kX>
static void norm_fwd_of(const FwdArgs &a, hipStream_t s) {
  if (a.cols <= 128) launch_fwd<T, R, kX, 16, 8>(a, s);
  else if (a.cols <= 512) launch_fwd<T, R, kX, 64, 8>(a, s);
  else if (a.cols <= 1024) launch_fwd<T, R, kX, 64, 16>(a, s);
  else if (a.cols <= 2048) launch_fwd<T, R, kX, 256, 8>(a, s);
  else if (a.cols <= 4096) launch_fwd<T, R, kX, 256, 16>(a, s);
  else if (a.cols <= 8192) launch_fwd<T, R, kX, 512, 16>(a, s);
  else if (a.cols <= 16384) launch_fwd<T, R, kX, 1024, 16>(a, s);
  else if (a.cols <= 32768) launch_fwd<T, R, kX, 1024, 32>(a, s);
  else hipLaunchKernelGGL((k_norm_fwd_wide<T, R, kX>), dim3(row_grid(a.rows)), dim3(1024), 0, s, a);
}

template <class T, class R, bool kX, bool kBias>
static void norm_bwd_of(const BwdArgs &a, const BwdPlan &p, hipStream_t s) {
  const dim3 g((uint32_t)p.lines);
#define TK_BWD(TPR, EPT)                                                                                         \
  hipLaunchKernelGGL((k_norm_bwd<T, R, kX, kBias, TPR, EPT>), g, dim3(TPR < 256 ? 256 : TPR), 0, s, a)
  if (p.tpr == 16) TK_BWD(16, 8);
  else if (p.tpr == 64 && p.ept == 8) TK_BWD(64, 8);
  else if (p.tpr == 64) TK_BWD(64, 16);
  else if (p.tpr == 256 && p.ept == 8) TK_BWD(256, 8);
  else if (p.tpr == 256) TK_BWD(256, 16);
  else if (p.tpr == 512) TK_BWD(512, 16);
  else TK_BWD(1024, 16);
#undef TK_BWD
}

template <class T, class R, bool kNorm, bool kX, bool kBias>
static void cols_bwd_of(const BwdArgs &a, const BwdPlan &p, hipStream_t s) {
  hipLaunchKernelGGL((k_cols_bwd<T, R, kNorm, kX, kBias>), dim3((uint32_t)p.strips, (uint32_t)p.lines), dim3(256), 0, s, a);
}

template <class T, class R>
struct RowKernels {
  static void norm_fwd(const FwdArgs &a, hipStream_t s) {
    if (a.x) norm_fwd_of<T, R, true>(a, s);
    else norm_fwd_of<T, R, false>(a, s);
  }
  static void norm_bwd(const BwdArgs &a, const BwdPlan &p, bool bias, hipStream_t s) {
    if (p.tpr == 0) {  // wide rows
      hipLaunchKernelGGL((k_row_stats<T, R>), dim3(row_grid(a.rows)), dim3(1024), 0, s, a);
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
  static void add_fwd(const AddArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((k_drop_add<T, R, std::is_same<T, float>::value, kChunk<T, R>, T>), dim3((a.chunks + 255) / 256),
                       dim3(256), 0, s, a);
  }
  static void add_bwd(const AddArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((k_drop_add<R, T, std::is_same<T, float>::value, kChunk<T, R>, T>), dim3((a.chunks + 255) / 256),
                       dim3(256), 0, s, a);
  }
  static RowTable table() { return {kChunk<T, R>, norm_fwd, norm_bwd, add_bwd_sums, add_fwd, add_bwd}; }
};

}  // namespace tk
