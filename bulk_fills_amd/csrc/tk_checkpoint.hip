// tk_checkpoint.hip -- activations kept in 8 bits: packing by stochastic rounding, and restoring.
// The backward passes that read the codes are the row operators' (tk_rows.h).
#include "tk_row_checks.h"
#include "tk_rows.h"

namespace tk {

struct CodeArgs {
  const void *x;
  void *y;
  int8_t *codes;
  float *scales;
  uint64_t row0, ldx, ldy, ldc;
  uint32_t cols, blocks, chunks, chunks_per_row, hk, start;
  Divisor per_row;  // chunks_per_row
};

constexpr int kCodes = 8;  // codes of a lane, so that sixteen lanes hold a block

// nv of a lane's elements, the others 0: fewer than all are loaded one by one.
template <class R>
__device__ __forceinline__ void load_lane(const R *p, int nv, float *v) {
  if (nv >= kCodes) {
    unpack<kCodes, R>(load_chunk<true, kCodes>(p), kCodes, v);
  } else {
#pragma unroll
    for (int e = 0; e < kCodes; ++e) v[e] = e < nv ? (float)p[e] : 0.0f;
  }
}

// Blocks whose largest element is below this are zeros: the quotient 127 / m stays finite, and the
// scale normal.
constexpr float kLeastHeld = 0x1p-100f;

// The float |x| times the float 127 / m lies on a grid that t - floor(t) is exact on, so a code is a
// comparison of two exact numbers: any evaluation of the definition gives the same one.  The largest
// magnitude is taken among the bit patterns, where NaN is above infinity.
template <class R>
__global__ __launch_bounds__(256) void k_checkpoint(CodeArgs a) {
  const uint32_t n = blockIdx.x * 256u + threadIdx.x;
  if (n >= a.chunks) return;  // whole blocks of sixteen lanes
  const uint32_t r = a.per_row.of(n), k = n - r * a.chunks_per_row, c = k * kCodes;
  const uint64_t row = a.row0 + r;
  const int nv = (int)(a.cols - c);
  float x[kCodes];
  load_lane<R>((const R *)a.x + row * a.ldx + c, nv, x);
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < kCodes; ++e) {
    const uint32_t b = __float_as_uint(x[e]) & 0x7FFFFFFFu;
    top = b > top ? b : top;
  }
  const auto larger = [&](uint32_t o) { top = o > top ? o : top; };
  larger(__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, true));   // quad_perm 1,0,3,2
  larger(__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, true));   // quad_perm 2,3,0,1
  larger(__builtin_amdgcn_update_dpp(0, (int)top, 0x141, 0xF, 0xF, true));  // row_half_mirror
  larger(__builtin_amdgcn_update_dpp(0, (int)top, 0x140, 0xF, 0xF, true));  // row_mirror
  const float m = __uint_as_float(top);
  const bool finite = top < 0x7F800000u, held = finite && m >= kLeastHeld;
  const float inverse = held ? __fdiv_rn(127.0f, m) : 0.0f;
  if (k % 16 == 0) a.scales[row * a.blocks + k / 16] = !finite ? __uint_as_float(0x7FC00000u) : held ? __fdiv_rn(m, 127.0f) : 0.0f;
  if (nv <= 0) return;
  uint32_t w[kCodes];
  chunk_words<kCodes>(a.hk, a.start + (uint32_t)row * a.cols + c, w);
  Chunk<int8_t, kCodes> code;
#pragma unroll
  for (int e = 0; e < kCodes; ++e) {
    const float t = held ? __builtin_fabsf(x[e]) * inverse : 0.0f, down = __builtin_floorf(t);
    const float up = tk_unit23(w[e]) < t - down ? 1.0f : 0.0f;
    code[e] = (int8_t)__builtin_copysignf(fminf(down + up, 127.0f), x[e]);
  }
  int8_t *out = a.codes + row * a.ldc + c;
  if (nv >= kCodes) {
    __builtin_nontemporal_store(code, (Chunk<int8_t, kCodes> *)out);
  } else {
#pragma unroll
    for (int e = 0; e < kCodes; ++e)
      if (e < nv) out[e] = code[e];
  }
}

template <class R>
__global__ __launch_bounds__(256) void k_restore(CodeArgs a) {
  const uint32_t n = blockIdx.x * 256u + threadIdx.x;
  if (n >= a.chunks) return;
  const uint32_t r = a.per_row.of(n), c = (n - r * a.chunks_per_row) * kCodes;
  const uint64_t row = a.row0 + r;
  const int nv = (int)(a.cols - c);
  float v[kCodes];
  load_lane<int8_t>(a.codes + row * a.ldc + c, nv, v);
  const float scale = a.scales[row * a.blocks + c / kCodeBlock];
#pragma unroll
  for (int e = 0; e < kCodes; ++e) v[e] *= scale;
  store_chunk<kCodes>((R *)a.y + row * a.ldy + c, nv, v);
}

// A call of more than 2^30 chunks is cut.
static tk_status run_codes(CodeArgs a, uint64_t rows, RowType t, bool r32, hipStream_t s) {
  const bool pack = a.x != nullptr;
  a.blocks = (a.cols + kCodeBlock - 1) / kCodeBlock;
  a.chunks_per_row = pack ? a.blocks * (kCodeBlock / kCodes) : (a.cols + kCodes - 1) / kCodes;
  a.per_row = Divisor(a.chunks_per_row);
  const uint64_t rows_each = (1ull << 30) / a.chunks_per_row;
  for (uint64_t r = 0; r < rows; r += rows_each) {
    a.row0 = r;
    a.chunks = (uint32_t)((rows - r < rows_each ? rows - r : rows_each) * a.chunks_per_row);
    const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((a.chunks + 255) / 256), dim3(256), 0, s, a); };
    if (t == kF32 || r32) go(pack ? k_checkpoint<float> : k_restore<float>);
    else if (t == kF16) go(pack ? k_checkpoint<f16_t> : k_restore<f16_t>);
    else go(pack ? k_checkpoint<bf16_t> : k_restore<bf16_t>);
    const tk_status st = launch_status();
    if (st != TK_OK) return st;
  }
  return TK_OK;
}

static uint64_t scales_of(uint64_t rows, uint64_t cols) { return rows * ((cols + kCodeBlock - 1) / kCodeBlock); }

static tk_status checkpoint(RowType t, uint32_t key, uint64_t start, uint64_t rows, uint64_t cols, uint32_t flags,
                            const void *x, uint64_t ldx, int8_t *codes, uint64_t ldc, float *scales, hipStream_t stream) {
  // every element has a draw: the counters' range holds as for dropout with p > 0
  tk_status st = check_scalars(start, rows, cols, 0.5f, 0.0f, flags, TK_RESIDUAL_F32);
  if (st != TK_OK || rows == 0 || cols == 0) return st;
  Arguments c{t, rows, cols, flags};
  c.matrix(x, ldx, c.res(), false, true);
  c.matrix_of(codes, rows, cols, ldc, 1, true, true, 2);
  c.vector(scales, scales_of(rows, cols), 4, true, true);
  if ((st = c.done()) != TK_OK) return st;
  CodeArgs a{};
  a.x = x; a.ldx = ldx; a.codes = codes; a.ldc = ldc; a.scales = scales; a.cols = (uint32_t)cols;
  a.hk = host_lowbias32(key);
  a.start = (uint32_t)start;
  return run_codes(a, rows, t, flags & TK_RESIDUAL_F32, stream);
}

static tk_status restore(RowType t, uint64_t rows, uint64_t cols, uint32_t flags, const int8_t *codes, uint64_t ldc,
                         const float *scales, void *y, uint64_t ldy, hipStream_t stream) {
  tk_status st = check_scalars(0, rows, cols, 0.0f, 0.0f, flags, TK_RESIDUAL_F32);
  if (st != TK_OK || rows == 0 || cols == 0) return st;
  Arguments c{t, rows, cols, flags};
  c.matrix_of(codes, rows, cols, ldc, 1, false, true, 2);
  c.vector(scales, scales_of(rows, cols), 4, false, true);
  c.matrix(y, ldy, c.res(), true, true);
  if ((st = c.done()) != TK_OK) return st;
  CodeArgs a{};
  a.codes = const_cast<int8_t *>(codes); a.ldc = ldc; a.scales = const_cast<float *>(scales); a.y = y; a.ldy = ldy;
  a.cols = (uint32_t)cols;
  return run_codes(a, rows, t, flags & TK_RESIDUAL_F32, stream);
}

}  // namespace tk

extern "C" {

#define TK_CHECKPOINT(SUFFIX, TYPE)                                                                                      \
  tk_status tk_checkpoint_##SUFFIX(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, uint32_t flags,      \
                                   const void *x, uint64_t ldx, int8_t *codes, uint64_t ldc, float *scales,              \
                                   hipStream_t stream) {                                                                 \
    return tk::checkpoint(TYPE, key, start_draw, rows, cols, flags, x, ldx, codes, ldc, scales, stream);                 \
  }                                                                                                                      \
  tk_status tk_checkpoint_restore_##SUFFIX(uint64_t rows, uint64_t cols, uint32_t flags, const int8_t *codes,            \
                                           uint64_t ldc, const float *scales, void *y, uint64_t ldy,                     \
                                           hipStream_t stream) {                                                         \
    return tk::restore(TYPE, rows, cols, flags, codes, ldc, scales, y, ldy, stream);                                     \
  }

TK_CHECKPOINT(f32, tk::kF32)
TK_CHECKPOINT(f16, tk::kF16)
TK_CHECKPOINT(bf16, tk::kBF16)

}  // extern "C"
