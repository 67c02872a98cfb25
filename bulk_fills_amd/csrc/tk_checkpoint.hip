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

constexpr int kPack = 16;  // elements of a lane of k_checkpoint: eight lanes hold a block
constexpr int kBlockLanes = kCodeBlock / kPack;

// Blocks whose largest element is below this are zeros: the quotient 127 / m stays finite, and the
// scale normal.
constexpr float kLeastHeld = 0x1p-100f;

// m / 127 to the nearest: a product with the rounded reciprocal and one correction, which is enough
// for a reciprocal that is itself the nearest (m at least kLeastHeld: nothing is subnormal).
__device__ __forceinline__ float over_127(float m) {
  const float r = 1.0f / 127.0f, q = m * r;
  return __builtin_fmaf(__builtin_fmaf(-q, 127.0f, m), r, q);
}

// floor(-x), and a << 1 plus b.
__device__ __forceinline__ int floor_of_negative(float x) {
  int n;
  asm("v_cvt_flr_i32_f32_e64 %0, -%1" : "=v"(n) : "v"(x));
  return n;
}
__device__ __forceinline__ uint32_t twice_and(uint32_t a, uint32_t b) {
  uint32_t n;
  asm("v_lshl_add_u32 %0, %1, 1, %2" : "=v"(n) : "v"(a), "v"(b));
  return n;
}

// The number whose highest byte is a code's magnitude below 0, from its word and t 2^24.
__device__ __forceinline__ uint32_t numbered(uint32_t word, float t) {
  return twice_and(word & 0x7FFFFFu, (uint32_t)floor_of_negative(t));
}

// Four codes from numbers that hold -|code| in their highest byte: those of negative elements (0xFF in
// `sign`) are the bytes themselves.  With the sign bit turned a byte is 128 - |code|, so that four are
// subtracted from 128 at once and none borrows.  A magnitude of 128 sets a highest bit in `over`.
__device__ __forceinline__ uint32_t four_codes(const uint32_t *n, uint32_t sign, uint32_t &over) {
  const uint32_t low = __builtin_amdgcn_perm(n[1], n[0], 0x0C0C0703), high = __builtin_amdgcn_perm(n[3], n[2], 0x07030C0C);
  const uint32_t negative = low | high, positive = 0x80808080u - (negative ^ 0x80808080u);
  over |= positive;
  return (negative & sign) | (positive & ~sign);
}

// Codes of 0x80, which no other magnitude than 128 gives, to 127 of their sign.
__device__ __forceinline__ uint32_t down_to_127(uint32_t codes, uint32_t sign) {
  const uint32_t x = codes ^ 0x80808080u, one = (~(((x & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | x) & 0x80808080u) >> 7;
  return codes + (one & sign) - (one & ~sign);
}

// Fewer than a lane's elements are loaded one by one, the others are 0.  Loads go through the caches at any
// size: a lane's vectors lie beside each other, so past them each line is read again for every vector
// (float 16384x8192 154 us instead of 113).
//
// A lane's elements as they are kept: their values, the largest magnitude's bits as a float's, and
// 0xFF in the byte of each negative one of four.
template <class R>
struct Lane {
  float x[kPack];
  __device__ __forceinline__ void load(const R *p, int nv) {
    if (nv >= kPack) {
      unpack<kPack, R>(load_chunk<false, kPack>(p), kPack, x);
    } else {
#pragma unroll
      for (int e = 0; e < kPack; ++e) x[e] = e < nv ? (float)p[e] : 0.0f;
    }
  }
  __device__ __forceinline__ float value(int e) const { return x[e]; }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;
#pragma unroll
    for (int e = 0; e < kPack; ++e) {
      const uint32_t b = __float_as_uint(x[e]) & 0x7FFFFFFFu;
      t = b > t ? b : t;
    }
    return t;
  }
  __device__ __forceinline__ uint32_t signs(int e) const {
    const uint32_t low = __builtin_amdgcn_perm(__float_as_uint(x[e + 1]), __float_as_uint(x[e]), 0x0C0C0B09);
    return low | __builtin_amdgcn_perm(__float_as_uint(x[e + 3]), __float_as_uint(x[e + 2]), 0x0B090C0C);
  }
};

// bfloat16: two elements to a register, whose magnitudes compare as 16-bit numbers.
template <>
struct Lane<bf16_t> {
  typedef uint32_t Pairs __attribute__((ext_vector_type(kPack / 2), aligned(2)));
  Pairs x;
  __device__ __forceinline__ void load(const bf16_t *p, int nv) {
    if (nv >= kPack) {
      x = *(const Pairs *)p;
    } else {
      const uint16_t *q = (const uint16_t *)p;
#pragma unroll
      for (int e = 0; e < kPack; e += 2) x[e / 2] = (e < nv ? (uint32_t)q[e] : 0u) | (e + 1 < nv ? (uint32_t)q[e + 1] << 16 : 0u);
    }
  }
  __device__ __forceinline__ float value(int e) const {
    return __uint_as_float(e % 2 ? x[e / 2] & 0xFFFF0000u : x[e / 2] << 16);
  }
  __device__ __forceinline__ uint32_t top() const {
    typedef uint16_t Two __attribute__((ext_vector_type(2)));
    Two t = 0;
#pragma unroll
    for (int i = 0; i < kPack / 2; ++i) t = __builtin_elementwise_max(t, __builtin_bit_cast(Two, x[i] & 0x7FFF7FFFu));
    return (uint32_t)(t[0] > t[1] ? t[0] : t[1]) << 16;
  }
  __device__ __forceinline__ uint32_t signs(int e) const {
    return __builtin_amdgcn_perm(x[e / 2 + 1], x[e / 2], 0x0B0A0908);
  }
};

// The float |x| times the float 127 / m lies on a grid that t - floor(t) is exact on, so a code is a
// comparison of two exact numbers: any evaluation of the definition gives the same one.  Here, with
// k = u 2^23 and N = floor(-t 2^24), -|code| = floor((N + 2 k) / 2^24): that is -floor(t) - 1 where 2 k is
// below ceil(t 2^24) - 2^24 floor(t), so below t's fraction, and -floor(t) elsewhere.
// The largest magnitude is taken among the bit patterns, where NaN is above infinity.
//
// Bound by memory and by its instructions alike, as only 3 bytes move for an element: bf16 16384x8192 72 us,
// 5.6 TB/s, of which 57 are the time of its 273 vector instructions a wave (17 an element).  Sixteen elements to
// a lane share what a lane does once: with eight, and each code's sign and rounding apart, 99 us.
//
// kWide: a wave takes 64 chunks of one row, so that rows and their addresses are the scalar unit's;
// else the chunks of all rows follow each other.  From 64 chunks on, which gains 2 % on long rows and loses
// where the row's last wave has many lanes idle.  us, wide and chunk by chunk, 2^25 elements but for the last:
//      columns    1024       1152       1280       1536       2048    16384x8192
//      bf16    18.4 18.2  28.5 18.2  26.1 18.3  22.6 18.3  18.5 18.3  72.2 73.7
//      f32     30.8 30.8  32.8 30.7  31.3 30.8  31.0 30.8  30.7 30.8   114  114
template <class R, bool kWide>
__global__ __launch_bounds__(256) void k_checkpoint(CodeArgs a) {
  uint32_t n = blockIdx.x * 256u + threadIdx.x, r, k;
  if constexpr (kWide) {
    n = blockIdx.x * 4u + (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (n >= a.chunks) return;  // here waves' worth of chunks
    r = a.per_row.of(n);
    k = (n - r * a.chunks_per_row) * 64 + (threadIdx.x & 63);
  } else {
    if (n >= a.chunks) return;  // whole blocks of a row's lanes
    r = a.per_row.of(n);
    k = n - r * a.chunks_per_row;
  }
  const uint64_t row = a.row0 + r;
  const uint32_t c = k * kPack;
  const int nv = (int)(a.cols - c);
  Lane<R> x;
  x.load((const R *)a.x + row * a.ldx + c, nv);
  uint32_t top = x.top();
  const auto larger = [&](uint32_t o) { top = o > top ? o : top; };
  larger(__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, true));  // quad_perm 1,0,3,2
  larger(__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, true));  // quad_perm 2,3,0,1
  if (kBlockLanes == 8) larger(__builtin_amdgcn_update_dpp(0, (int)top, 0x141, 0xF, 0xF, true));  // row_half_mirror
  if (nv <= 0) return;
  const float m = __uint_as_float(top);
  const bool finite = top < 0x7F800000u, held = finite && m >= kLeastHeld;
  if (k % kBlockLanes == 0)
    a.scales[row * a.blocks + k / kBlockLanes] = !finite ? __uint_as_float(0x7FC00000u) : held ? over_127(m) : 0.0f;
  const float inverse = held ? __fdiv_rn(127.0f, m) : 0.0f;
  uint32_t w[kPack];
  chunk_words<kPack>(a.hk, a.start + (uint32_t)row * a.cols + c, w);
  // One product gives t 2^24 where 2^24 inverse is finite and no t is rounded to 0: where t is subnormal
  // the product may differ from t 2^24, but both are above 0 and below 1.
  if (__all(!held || (m >= 0x1p-96f && m < 127.0f))) {
#pragma unroll
    for (int e = 0; e < kPack; ++e)
      w[e] = numbered(w[e], __builtin_fabsf(x.value(e)) * (inverse * 0x1p24f));
  } else {
#pragma unroll
    for (int e = 0; e < kPack; ++e) w[e] = numbered(w[e], __builtin_fabsf(x.value(e)) * inverse * 0x1p24f);
  }
  typedef uint32_t Codes __attribute__((ext_vector_type(kPack / 4), aligned(1)));
  Codes code;
  uint32_t over = 0;
#pragma unroll
  for (int e = 0; e < kPack; e += 4) code[e / 4] = four_codes(w + e, x.signs(e), over);
  // The largest t lies up to two units of its last place above 127, and is rounded up then once in 2^16.
  if (__any(over & 0x80808080u))
#pragma unroll
    for (int e = 0; e < kPack; e += 4) code[e / 4] = down_to_127(code[e / 4], x.signs(e));
  if (!__all(finite)) code = finite ? code : Codes(0);
  int8_t *out = a.codes + row * a.ldc + c;
  if (nv >= kPack) {
    __builtin_nontemporal_store(code, (Codes *)out);
  } else {
#pragma unroll
    for (int e = 0; e < kPack; ++e)
      if (e < nv) out[e] = (int8_t)(code[e / 4] >> (8 * (e % 4)));
  }
}

// A lane takes V chunks, 64 apart, each 16 bytes of y: four of 16-bit elements, two of floats (16384x8192 with
// one, two and four: bf16 69.8, 67.7 and 65.2 us, float 124, 104 and 112).  kWide as above (V = 1 where it is
// not): chunk by chunk the bf16 69.8 and float 123 us; 2^25 elements at 512 to 4096 columns within 1 % either way,
// but bf16 at 512 (17.9 for 17.0).
template <class R, int CH, bool kWide, int V>
__global__ __launch_bounds__(256) void k_restore(CodeArgs a) {
  uint32_t n = blockIdx.x * 256u + threadIdx.x, r, c;
  if constexpr (kWide) {
    n = blockIdx.x * 4u + (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (n >= a.chunks) return;
    r = a.per_row.of(n);
    c = ((n - r * a.chunks_per_row) * (64 * V) + (threadIdx.x & 63)) * CH;
  } else {
    if (n >= a.chunks) return;
    r = a.per_row.of(n);
    c = (n - r * a.chunks_per_row) * CH;
  }
  const uint64_t row = a.row0 + r;
  Codes<CH> codes[V];
  float scale[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t at = c + j * 64 * CH;
    codes[j].template load<false>(a.codes + row * a.ldc + chunk_at<CH>(at, a.cols));
    scale[j] = a.scales[row * a.blocks + (at < a.cols ? at / kCodeBlock : a.blocks - 1)];
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t at = c + j * 64 * CH;
    const int nv = (int)(a.cols - at);
    const float by = held_scale(scale[j]);
    float v[CH];
    codes[j].floats(nv, v);
#pragma unroll
    for (int e = 0; e < CH; ++e) v[e] *= by;
    if (nv > 0) store_chunk<CH>((R *)a.y + row * a.ldy + at, nv, v);
  }
}

// A call of more than 2^30 chunks (waves of them, where rows have 64 and more) is cut.
static tk_status run_codes(CodeArgs a, uint64_t rows, RowType t, bool r32, hipStream_t s) {
  const bool pack = a.x != nullptr;
  const uint32_t whole = t == kF32 || r32 ? 4 : 8, ch = a.cols < whole ? 1 : whole;  // k_restore's chunk
  const uint32_t beside = whole / 2;                                                // and chunks of a lane
  a.blocks = (a.cols + kCodeBlock - 1) / kCodeBlock;
  a.chunks_per_row = pack ? a.blocks * kBlockLanes : (a.cols + ch - 1) / ch;
  const bool wide = a.chunks_per_row >= 64;
  if (wide) a.chunks_per_row = pack ? (a.chunks_per_row + 63) / 64 : (a.chunks_per_row + 64 * beside - 1) / (64 * beside);
  a.per_row = Divisor(a.chunks_per_row);
  const uint64_t rows_each = (wide ? 1ull << 25 : 1ull << 30) / a.chunks_per_row;
  for (uint64_t r = 0; r < rows; r += rows_each) {
    a.row0 = r;
    a.chunks = (uint32_t)((rows - r < rows_each ? rows - r : rows_each) * a.chunks_per_row);
    const auto go = [&](auto kernel, uint32_t each) {
      hipLaunchKernelGGL(kernel, dim3((a.chunks + each - 1) / each), dim3(256), 0, s, a);
    };
    const auto type = [&](auto h) {
      typedef decltype(h) R;
      constexpr int CH = 16 / sizeof(R);
      if (pack && wide) go(k_checkpoint<R, true>, 4);
      else if (pack) go(k_checkpoint<R, false>, 256);
      else if (wide) go(k_restore<R, CH, true, CH / 2>, 4);
      else if (ch == 1) go(k_restore<R, 1, false, 1>, 256);
      else go(k_restore<R, CH, false, 1>, 256);
    };
    if (whole == 4) type(float());
    else if (t == kF16) type(f16_t());
    else type(bf16_t());
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
