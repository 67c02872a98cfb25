// tk_rows.hip -- entry points of the row operators: how a backward call is cut, and the kernel
// that adds up the partial column sums.
#include "tk_row_checks.h"

namespace tk {

// ---------------------------------------------------------------------------------------
// The end of the column sums: lines of partial sums into element type float or the parameters',
// in a fixed order
// ---------------------------------------------------------------------------------------
// Up to this many lines four waves of k_finish add up, more sixteen (fused backward bf16
// 512x24576, of 5 lines, 31.4 us, with sixteen waves 32.7; layer norm's 40x32768 11.8 and 13.0).
constexpr uint64_t kFewLines = 16;

struct FinishArgs {
  const float *partial;
  void *out[3];  // null: not wanted
  uint64_t lines;
  uint32_t cols, col0;  // col0: the launch's first column
  int kind;             // 0 float, 1 binary16, 2 bfloat16
};

// A work-group takes kCols columns, a wave 64 / kCols lines of them at a time: 64, or 32 up to
// 4096 columns, where work-groups are few (layer norm backward bf16 1000x2048: 11.1 us, with 64
// columns 11.5; 300x12000 with sixteen waves 15.1 and 14.2).
//
// The sum of every kLines-th of a column's lines from the first one, at most kSteps of them.  All
// are read at once, beyond the last line that line again: a loop over the lines waits for loads
// one by one (2000x1024, of 250 lines: 9.2 against 12.9 us).  Several lines have fewer than 2^18
// columns: the distances fit 32 bits.
template <int kLines, int kSteps>
__device__ __forceinline__ float column_sum(const float *p, uint32_t first, uint32_t lines, uint32_t pitch) {
  float v[kSteps], s = 0.0f;
  uint32_t at = first * pitch;
  const uint32_t last = (lines - 1) * pitch;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    v[i] = __builtin_nontemporal_load(p + (at < last ? at : last));
    at += kLines * pitch;
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) s += first + kLines * i < lines ? v[i] : 0.0f;
  return s;
}

template <int kCols, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void k_finish(FinishArgs a) {
  constexpr uint32_t kLines = 64 * kWaves / kCols;
  constexpr int kMost = (kWaves == 16 ? kMaxLines : kFewLines) / kLines;
  __shared__ float part[kWaves][kCols];
  void *out = a.out[blockIdx.y];
  if (!out) return;
  const uint32_t i = threadIdx.x % kCols, first = threadIdx.x / kCols, c = a.col0 + blockIdx.x * kCols + i;
  if (c < a.cols) {
    const uint32_t lines = (uint32_t)a.lines, pitch = (uint32_t)line_pitch(a.cols);
    const float *p = a.partial + (uint64_t)blockIdx.y * lines * pitch + c;
    float s;
    if (lines == 0) s = 0.0f;  // no rows, no workspace
    else if (lines <= kLines) s = column_sum<kLines, 1>(p, first, lines, pitch);
    else if (lines <= 2 * kLines) s = column_sum<kLines, 2>(p, first, lines, pitch);
    else if (kMost == 4 || lines <= 4 * kLines) s = column_sum<kLines, 4>(p, first, lines, pitch);
    else if (kMost == 8 || lines <= 8 * kLines) s = column_sum<kLines, 8>(p, first, lines, pitch);
    else s = column_sum<kLines, 16>(p, first, lines, pitch);
    if (kCols == 32) s += __shfl_xor(s, 32);
    part[threadIdx.x >> 6][i] = s;
  }
  __syncthreads();
  if (threadIdx.x < kCols && c < a.cols) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) s += part[w][i];
    if (a.kind == 0) ((float *)out)[c] = s;
    else if (a.kind == 1) ((_Float16 *)out)[c] = (_Float16)s;
    else ((__bf16 *)out)[c] = (__bf16)s;
  }
}

// ---------------------------------------------------------------------------------------
// How a backward call is cut
// ---------------------------------------------------------------------------------------
constexpr uint64_t kRowsInRegisters = 8192;      // columns that k_norm_bwd holds

// Up to this many sets of rows one work-group (or one to a strip) takes them all and writes the
// gradients itself (layer norm backward bf16 128x128 5.1 us, with a second kernel 6.4; four sets
// to a work-group take up to 3 us longer than one with that kernel).  Calls that want no column sums
// (`sums` false) have nothing to gain by few work-groups: layer norm backward bf16 2x8192 3.6 us
// with two and 4.5 with one, 256x8192 4.3 us with 256 and 7.0 with 64.
constexpr uint64_t kAloneSets = 2;

// Partial sums of this many floats or more (of one gradient) are written past the caches: the
// second kernel starts when they are out of the L2s (layer norm backward bf16 300x8192 12.2 us,
// through them 12.9; 1000x4096 12.6 and 13.5).  Fewer are read from there (8000x2048 22.0 us,
// past them 22.6).
constexpr uint64_t kPastFloats = 9 << 16;

// Strips of columns by sets of rows: one work-group of 16 waves a compute unit, or fewer that
// have one row for each of their groups of lanes.  Dropout-add's backward bf16 8192x4096 takes
// 25.9, 26.8, 28.3 and 28.8 us with 256, 512, 768 and 1024 work-groups, the fused backward
// 512x24576 31.8, 33.0, 35.2 and 38.2.
static BwdPlan strips_plan(int chunk, uint64_t rows, uint64_t cols, bool sums) {
  BwdPlan p{};
  const int ch = cols < (uint64_t)chunk ? 1 : chunk;
  p.lanes = cols <= 8ull * ch ? 8 : cols <= 16ull * ch ? 16 : cols <= 32ull * ch ? 32 : 64;
  p.strips = (cols + p.lanes * ch - 1) / (p.lanes * ch);
  const uint64_t at_once = 16 * 64 / p.lanes, most = (rows + at_once - 1) / at_once;
  p.lines = sums && most <= kAloneSets ? 1 : p.strips < kMaxLines ? kMaxLines / p.strips : 1;
  if (p.lines > most) p.lines = most;
  p.room = p.lines;
  return p;
}

// Layer norm's: one work-group of up to 16 waves to a compute unit, as many rows at a time as
// it has waves for, so that there are few lines of partial sums (fused backward bf16 8192x4096:
// 68 us with two rows of eight waves to a work-group, 79 with one row and twice the lines).
// Beyond 8192 columns the column sums do not fit the registers beside a row: two kernels and a
// second read of dy and sum are faster (fused backward bf16 4096x16384: 160 against 286 us).
static BwdPlan norm_plan(int chunk, uint64_t rows, uint64_t cols, bool sums) {
  if (cols > kRowsInRegisters) return strips_plan(chunk, rows, cols, sums);
  BwdPlan p{};
  p.lanes = cols <= 64 ? 8 : cols <= 128 ? 16 : cols <= 256 ? 32 : 64;
  p.row_waves = p.lanes < 64 ? 1 : (int)((cols + 511) / 512);
  p.waves = 16 / p.row_waves * p.row_waves;
  const uint64_t per = p.lanes < 64 ? 64 * p.waves / p.lanes : p.waves / p.row_waves, sets = (rows + per - 1) / per;
  // What a set reads and what its line costs to write and read are alike: wide rows go several
  // sets to a work-group (256x8192 with 256, 128 and 64 lines: 17.9, 13.0 and 12.4 us).
  uint64_t least = sums && sets <= kAloneSets ? sets : 1;
  while (sums && sets > kAloneSets && least < 4 && sets * cols >= (least * least) << 19) least *= 2;
  p.lines = (sets + least - 1) / least;
  if (p.lines > kMaxLines) p.lines = kMaxLines;
  p.room = sets < kMaxLines ? sets : kMaxLines;
  return p;
}

// Room for at least the plan's lines, and never less for more rows: a caller with batches of many
// sizes keeps what the largest needs.
static uint64_t bytes_of(const BwdPlan &p, uint64_t cols) { return p.lines > 1 ? 12 * p.room * line_pitch(cols) : 0; }

// The larger of both chunk sizes and both kinds of call, so that one size serves every type.
static uint64_t workspace_bytes(uint64_t rows, uint64_t cols) {
  if (rows == 0 || cols == 0) return 0;
  uint64_t b = 0;
  for (int chunk = 4; chunk <= 8; chunk += 4) {
    const uint64_t s = bytes_of(strips_plan(chunk, rows, cols, true), cols), n = bytes_of(norm_plan(chunk, rows, cols, true), cols);
    b = s > b ? s : b;
    b = n > b ? n : b;
  }
  return b + (cols > kRowsInRegisters ? 8 * rows : 0);
}

constexpr uint32_t kRowFlags = TK_RESIDUAL_F32 | TK_PARAMS_F32;

static RowTable table_of(RowType t, uint32_t flags) {
  const bool r32 = flags & TK_RESIDUAL_F32;
  switch (t) {
    case kF16: return r32 ? rows_f16_r32() : rows_f16();
    case kBF16: return r32 ? rows_bf16_r32() : rows_bf16();
    default: return rows_f32();
  }
}

tk_status finish(RowType t, uint32_t flags, const float *partial, uint64_t lines, uint64_t cols, void *a, void *b,
                        void *c, hipStream_t stream) {
  FinishArgs f{partial, {a, b, c}, lines, (uint32_t)cols, 0, params_f32(t, flags) ? 0 : t == kF16 ? 1 : 2};
  const uint64_t wide = lines <= kFewLines || cols > 4096 ? 64 : 32;
  const uint64_t most = 1ull << 26;  // columns of a launch, which holds fewer than 2^32 threads
  for (uint64_t k = 0; k < cols; k += most) {
    f.col0 = (uint32_t)k;
    const uint64_t n = cols - k < most ? cols - k : most;
    const dim3 grid((uint32_t)((n + wide - 1) / wide), c ? 3 : b ? 2 : 1);
    if (lines <= kFewLines) hipLaunchKernelGGL((k_finish<64, 4>), grid, dim3(256), 0, stream, f);
    else if (wide == 64) hipLaunchKernelGGL((k_finish<64, 16>), grid, dim3(1024), 0, stream, f);
    else hipLaunchKernelGGL((k_finish<32, 16>), grid, dim3(1024), 0, stream, f);
  }
  return launch_status();
}

// ---------------------------------------------------------------------------------------
// Dropout-add
// ---------------------------------------------------------------------------------------
// The element-wise launches.  A contiguous call is one long row (with a bias, if its rows are
// whole chunks).  A call of more than 2^30 chunks is cut.
static tk_status run_add(void (*launch)(const AddArgs &, int, hipStream_t), int chunk, AddArgs a, uint64_t rows, uint64_t cols,
                         int in_size, int out_size, hipStream_t stream) {
  const bool dense = rows == 1 || (a.ldx == cols && a.ldy == cols && (!a.residual || a.ldr == cols));
  a.flat = dense && rows * cols >= (uint64_t)chunk && (!a.bias || cols % chunk == 0);
  if (!a.flat && cols < (uint64_t)chunk) chunk = 1;  // no row holds a whole chunk
  const uint64_t per_row = (cols + chunk - 1) / chunk, most = 1ull << 30;  // chunks
  a.bias_cols = cols;
  if (!a.flat || a.bias) {
    a.chunks_per_row = (uint32_t)per_row;
    a.per_row = Divisor(per_row);
  }
  if (a.flat) {
    // pieces of whole rows where there is a bias, and none shorter than a chunk
    const uint64_t n = rows * cols, piece = a.bias ? most / per_row * cols : most * chunk;
    for (uint64_t k = 0, m; k < n; k += m) {
      AddArgs b = a;
      m = n - k < piece + chunk ? n - k : piece;
      b.x = (const char *)a.x + k * in_size;
      if (a.residual) b.residual = (const char *)a.residual + k * out_size;
      b.y = (char *)a.y + k * out_size;
      b.drop.start = a.drop.start + (uint32_t)k;
      b.chunks = (uint32_t)((m + chunk - 1) / chunk);
      b.cols64 = m;
      launch(b, chunk, stream);
      const tk_status st = launch_status();
      if (st != TK_OK) return st;
    }
    return TK_OK;
  }
  const uint64_t rows_each = most / per_row;
  a.cols64 = cols;
  for (uint64_t r = 0; r < rows; r += rows_each) {
    AddArgs b = a;
    b.row0 = r;
    b.chunks = (uint32_t)((rows - r < rows_each ? rows - r : rows_each) * per_row);
    launch(b, chunk, stream);
    const tk_status st = launch_status();
    if (st != TK_OK) return st;
  }
  return TK_OK;
}

static tk_status dropout_add(RowType t, uint32_t key, uint64_t start, uint64_t rows, uint64_t cols, float p, uint32_t flags,
                             const void *x, uint64_t ldx, const void *bias, const void *residual, uint64_t ldr, void *y,
                             uint64_t ldy, hipStream_t stream) {
  tk_status st = check_scalars(start, rows, cols, p, 0.0f, flags, kRowFlags);
  if (st != TK_OK || rows == 0 || cols == 0) return st;
  Arguments c{t, rows, cols, flags};
  c.matrix(x, ldx, c.t(), false, true);
  c.vector(bias, cols, c.par(), false, false);
  c.matrix(residual, ldr, c.res(), false, false);
  c.matrix(y, ldy, c.res(), true, true);
  if ((st = c.done()) != TK_OK) return st;
  AddArgs a{};
  a.x = x; a.ldx = ldx; a.bias = bias; a.residual = residual; a.ldr = ldr; a.y = y; a.ldy = ldy;
  a.params_f32 = params_f32(t, flags);
  a.drop = drop_of(key, start, p);
  a.once = rows * cols * (c.t() + (residual ? c.res() : 0)) > kCachedReads;
  const RowTable k = table_of(t, flags);
  return run_add(k.add_fwd, k.chunk, a, rows, cols, c.t(), c.res(), stream);
}

static tk_status dropout_add_backward(RowType t, uint32_t key, uint64_t start, uint64_t rows, uint64_t cols, float p,
                                      uint32_t flags, const void *dy, uint64_t lddy, void *dx, uint64_t lddx, void *dbias,
                                      void *workspace, uint64_t workspace_bytes_, hipStream_t stream) {
  tk_status st = check_scalars(start, rows, cols, p, 0.0f, flags, kRowFlags);
  if (st != TK_OK || cols == 0) return st;
  Arguments c{t, rows, cols, flags};
  if (rows == 0) {
    c.vector(dbias, cols, c.par(), true, false);
    if ((st = c.done()) != TK_OK || !dbias) return st;
    return finish(t, flags, nullptr, 0, cols, dbias, nullptr, nullptr, stream);
  }
  c.matrix(dy, lddy, c.res(), false, true);
  c.matrix(dx, lddx, c.t(), true, true);
  c.vector(dbias, cols, c.par(), true, false);
  const uint64_t need = dbias ? workspace_bytes(rows, cols) : 0;
  if (!serves(workspace, workspace_bytes_, need)) return TK_EINVAL;
  if (need) c.vector(workspace, need / 4, 4, true, true);
  if ((st = c.done()) != TK_OK) return st;
  const RowTable k = table_of(t, flags);
  if (!dbias) {
    AddArgs a{};
    a.x = dy; a.ldx = lddy; a.y = dx; a.ldy = lddx;
    a.drop = drop_of(key, start, p);
    a.once = rows * cols * c.res() > kCachedReads;
    return run_add(k.add_bwd, k.chunk, a, rows, cols, c.res(), c.t(), stream);
  }
  const BwdPlan plan = strips_plan(k.chunk, rows, cols, true);
  BwdArgs a{};
  a.dy = dy; a.lddy = lddy; a.dx = dx; a.lddx = lddx;
  a.rows = rows; a.cols = (uint32_t)cols;
  a.alone = plan.lines == 1;
  a.sums[2] = dbias;
  a.partial = a.alone ? nullptr : (float *)workspace;
  a.params_f32 = params_f32(t, flags);
  a.drop = drop_of(key, start, p);
  a.once = rows * cols * c.res() > kCachedReads;
  k.add_bwd_sums(a, plan, stream);
  if ((st = launch_status()) != TK_OK || a.alone) return st;
  return finish(t, flags, a.partial, plan.lines, cols, dbias, nullptr, nullptr, stream);
}

// ---------------------------------------------------------------------------------------
// Layer norm, alone and after dropout-add
// ---------------------------------------------------------------------------------------
// `fused`: x is needed and the norm's input is residual + drop(x + bias); else the norm's input
// comes as `residual`.
static tk_status norm_forward(RowType t, bool fused, uint32_t key, uint64_t start, uint64_t rows, uint64_t cols, float p,
                              float eps, uint32_t flags, const void *x, uint64_t ldx, const void *bias, const void *residual,
                              uint64_t ldr, const void *gamma, const void *beta, void *sum, uint64_t lds, void *y,
                              uint64_t ldy, float *mean, float *rstd, hipStream_t stream) {
  tk_status st = check_scalars(start, rows, cols, p, eps, flags, kRowFlags);
  if (st != TK_OK || rows == 0 || cols == 0) return st;
  Arguments c{t, rows, cols, flags};
  if (fused) c.matrix(x, ldx, c.t(), false, true);
  c.vector(bias, cols, c.par(), false, false);
  c.matrix(residual, ldr, c.res(), false, !fused);
  c.vector(gamma, cols, c.par(), false, false);
  c.vector(beta, cols, c.par(), false, false);
  c.matrix(sum, lds, c.res(), true, false);
  c.matrix(y, ldy, c.t(), true, true);
  c.vector(mean, rows, 4, true, false);
  c.vector(rstd, rows, 4, true, false);
  if ((st = c.done()) != TK_OK) return st;
  FwdArgs a{};
  a.x = x; a.ldx = ldx; a.bias = bias; a.residual = residual; a.ldr = ldr; a.gamma = gamma; a.beta = beta;
  a.sum = sum; a.lds = lds; a.y = y; a.ldy = ldy; a.mean = mean; a.rstd = rstd;
  a.rows = rows; a.cols = (uint32_t)cols; a.eps = eps;
  a.params_f32 = params_f32(t, flags);
  a.drop = drop_of(key, start, p);
  a.once = rows * cols * ((fused ? c.t() : 0) + (residual ? c.res() : 0)) > kCachedReads;
  table_of(t, flags).norm_fwd(a, stream);
  return launch_status();
}

// `kept`: `sum` is a checkpoint's codes, and `scales` theirs.
static tk_status norm_backward(RowType t, bool fused, uint32_t key, uint64_t start, uint64_t rows, uint64_t cols, float p,
                               uint32_t flags, const void *dy, uint64_t lddy, const void *dsum, uint64_t ldds,
                               const void *sum, uint64_t lds, bool kept, const float *scales, const void *gamma,
                               const float *mean, const float *rstd, void *dx, uint64_t lddx, void *dresidual,
                               uint64_t lddr, void *dgamma, void *dbeta, void *dbias, void *workspace,
                               uint64_t workspace_bytes_, hipStream_t stream) {
  tk_status st = check_scalars(start, rows, cols, p, 0.0f, flags, kRowFlags);
  if (st != TK_OK || cols == 0) return st;
  Arguments c{t, rows, cols, flags};
  const bool sums = dgamma || dbeta || dbias;
  if (rows == 0) {
    c.vector(dgamma, cols, c.par(), true, false);
    c.vector(dbeta, cols, c.par(), true, false);
    c.vector(dbias, cols, c.par(), true, false);
    if ((st = c.done()) != TK_OK || !sums) return st;
    return finish(t, flags, nullptr, 0, cols, dgamma, dbeta, dbias, stream);
  }
  c.matrix(dy, lddy, c.t(), false, true);
  c.matrix(dsum, ldds, c.res(), false, false);
  const uint64_t blocks = (cols + kCodeBlock - 1) / kCodeBlock;
  c.matrix(sum, lds, kept ? 1 : c.res(), false, true);
  if (kept) c.vector(scales, rows * blocks, 4, false, true);
  c.vector(gamma, cols, c.par(), false, false);
  c.vector(mean, rows, 4, false, true);
  c.vector(rstd, rows, 4, false, true);
  if (fused) c.matrix(dx, lddx, c.t(), true, true);
  c.matrix(dresidual, lddr, c.res(), true, !fused);
  c.vector(dgamma, cols, c.par(), true, false);
  c.vector(dbeta, cols, c.par(), true, false);
  c.vector(dbias, cols, c.par(), true, false);
  const uint64_t need = sums || cols > kRowsInRegisters ? workspace_bytes(rows, cols) : 0;
  if (!serves(workspace, workspace_bytes_, need)) return TK_EINVAL;
  if (need) c.vector(workspace, need / 4, 4, true, true);
  if ((st = c.done()) != TK_OK) return st;
  const RowTable k = table_of(t, flags);
  const BwdPlan plan = norm_plan(k.chunk, rows, cols, sums);
  BwdArgs a{};
  a.dy = dy; a.lddy = lddy; a.dsum = dsum; a.ldds = ldds; a.sum = sum; a.lds = lds;
  a.scales = kept ? scales : nullptr; a.blocks = (uint32_t)blocks;
  a.gamma = gamma; a.mean = mean; a.rstd = rstd;
  a.dx = dx; a.lddx = lddx; a.dresidual = dresidual; a.lddr = lddr;
  a.rows = rows; a.cols = (uint32_t)cols; a.waves = (uint32_t)plan.row_waves;
  a.alone = sums && plan.lines == 1;
  a.sums[0] = dgamma; a.sums[1] = dbeta; a.sums[2] = dbias;
  a.partial = sums && !a.alone ? (float *)workspace : nullptr;
  a.past = plan.lines * cols >= kPastFloats;
  a.stats = !plan.strips ? nullptr : (float *)((char *)workspace + need - 8 * rows);
  a.params_f32 = params_f32(t, flags);
  a.drop = drop_of(key, start, p);
  a.once = rows * cols * (c.t() + (dsum ? c.res() : 0) + (kept ? 1 : c.res())) > kCachedReads;
  k.norm_bwd(a, plan, dbias != nullptr, stream);
  if ((st = launch_status()) != TK_OK || !sums || a.alone) return st;
  return finish(t, flags, a.partial, plan.lines, cols, dgamma, dbeta, dbias, stream);
}

}  // namespace tk

extern "C" {

tk_status tk_backward_workspace_bytes(uint64_t rows, uint64_t cols, uint64_t *bytes) {
  if (!bytes) return TK_EINVAL;
  if (rows >= tk::kMaxDim || cols >= tk::kMaxDim) return TK_ERANGE;
  *bytes = tk::workspace_bytes(rows, cols);
  return TK_OK;
}

#define TK_ROW_OPERATORS(SUFFIX, TYPE)                                                                                   \
  tk_status tk_dropout_add_##SUFFIX(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p,            \
                                    uint32_t flags, const void *x, uint64_t ldx, const void *bias, const void *residual, \
                                    uint64_t ldr, void *y, uint64_t ldy, hipStream_t stream) {                           \
    return tk::dropout_add(TYPE, key, start_draw, rows, cols, p, flags, x, ldx, bias, residual, ldr, y, ldy, stream);    \
  }                                                                                                                      \
  tk_status tk_dropout_add_backward_##SUFFIX(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p,   \
                                             uint32_t flags, const void *dy, uint64_t lddy, void *dx, uint64_t lddx,     \
                                             void *dbias, void *workspace, uint64_t workspace_bytes,                     \
                                             hipStream_t stream) {                                                       \
    return tk::dropout_add_backward(TYPE, key, start_draw, rows, cols, p, flags, dy, lddy, dx, lddx, dbias, workspace,   \
                                    workspace_bytes, stream);                                                            \
  }                                                                                                                      \
  tk_status tk_layer_norm_##SUFFIX(uint64_t rows, uint64_t cols, float eps, uint32_t flags, const void *x, uint64_t ldx, \
                                   const void *gamma, const void *beta, void *y, uint64_t ldy, float *mean, float *rstd, \
                                   hipStream_t stream) {                                                                 \
    return tk::norm_forward(TYPE, false, 0, 0, rows, cols, 0.0f, eps, flags, nullptr, 0, nullptr, x, ldx, gamma, beta,   \
                            nullptr, 0, y, ldy, mean, rstd, stream);                                                     \
  }                                                                                                                      \
  tk_status tk_layer_norm_backward_##SUFFIX(uint64_t rows, uint64_t cols, uint32_t flags, const void *dy, uint64_t lddy, \
                                            const void *x, uint64_t ldx, const void *gamma, const float *mean,           \
                                            const float *rstd, void *dx, uint64_t lddx, void *dgamma, void *dbeta,       \
                                            void *workspace, uint64_t workspace_bytes, hipStream_t stream) {             \
    return tk::norm_backward(TYPE, false, 0, 0, rows, cols, 0.0f, flags, dy, lddy, nullptr, 0, x, ldx, false, nullptr,   \
                             gamma, mean, rstd, nullptr, 0, dx, lddx, dgamma, dbeta, nullptr, workspace,                 \
                             workspace_bytes, stream);                                                                   \
  }                                                                                                                      \
  tk_status tk_dropout_add_layer_norm_##SUFFIX(                                                                          \
      uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p, float eps, uint32_t flags,               \
      const void *x, uint64_t ldx, const void *bias, const void *residual, uint64_t ldr, const void *gamma,              \
      const void *beta, void *sum, uint64_t lds, void *y, uint64_t ldy, float *mean, float *rstd, hipStream_t stream) {  \
    return tk::norm_forward(TYPE, true, key, start_draw, rows, cols, p, eps, flags, x, ldx, bias, residual, ldr, gamma,  \
                            beta, sum, lds, y, ldy, mean, rstd, stream);                                                 \
  }                                                                                                                      \
  tk_status tk_dropout_add_layer_norm_backward_##SUFFIX(                                                                 \
      uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p, uint32_t flags, const void *dy,          \
      uint64_t lddy, const void *dsum, uint64_t ldds, const void *sum, uint64_t lds, const void *gamma,                  \
      const float *mean, const float *rstd, void *dx, uint64_t lddx, void *dresidual, uint64_t lddr, void *dgamma,       \
      void *dbeta, void *dbias, void *workspace, uint64_t workspace_bytes, hipStream_t stream) {                         \
    return tk::norm_backward(TYPE, true, key, start_draw, rows, cols, p, flags, dy, lddy, dsum, ldds, sum, lds, false,   \
                             nullptr, gamma, mean, rstd, dx, lddx, dresidual, lddr, dgamma, dbeta, dbias, workspace,     \
                             workspace_bytes, stream);                                                                   \
  }

#define TK_BACKWARD_FROM_CHECKPOINT(SUFFIX, TYPE)                                                                        \
  tk_status tk_layer_norm_backward_checkpoint_##SUFFIX(                                                                  \
      uint64_t rows, uint64_t cols, uint32_t flags, const void *dy, uint64_t lddy, const int8_t *codes, uint64_t ldc,    \
      const float *scales, const void *gamma, const float *mean, const float *rstd, void *dx, uint64_t lddx,             \
      void *dgamma, void *dbeta, void *workspace, uint64_t workspace_bytes, hipStream_t stream) {                        \
    return tk::norm_backward(TYPE, false, 0, 0, rows, cols, 0.0f, flags, dy, lddy, nullptr, 0, codes, ldc, true, scales, \
                             gamma, mean, rstd, nullptr, 0, dx, lddx, dgamma, dbeta, nullptr, workspace,                 \
                             workspace_bytes, stream);                                                                   \
  }                                                                                                                      \
  tk_status tk_dropout_add_layer_norm_backward_checkpoint_##SUFFIX(                                                      \
      uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p, uint32_t flags, const void *dy,          \
      uint64_t lddy, const void *dsum, uint64_t ldds, const int8_t *codes, uint64_t ldc, const float *scales,            \
      const void *gamma, const float *mean, const float *rstd, void *dx, uint64_t lddx, void *dresidual, uint64_t lddr,  \
      void *dgamma, void *dbeta, void *dbias, void *workspace, uint64_t workspace_bytes, hipStream_t stream) {           \
    return tk::norm_backward(TYPE, true, key, start_draw, rows, cols, p, flags, dy, lddy, dsum, ldds, codes, ldc, true,  \
                             scales, gamma, mean, rstd, dx, lddx, dresidual, lddr, dgamma, dbeta, dbias, workspace,      \
                             workspace_bytes, stream);                                                                   \
  }

TK_ROW_OPERATORS(f32, tk::kF32)
TK_ROW_OPERATORS(f16, tk::kF16)
TK_ROW_OPERATORS(bf16, tk::kBF16)
TK_BACKWARD_FROM_CHECKPOINT(f32, tk::kF32)
TK_BACKWARD_FROM_CHECKPOINT(f16, tk::kF16)
TK_BACKWARD_FROM_CHECKPOINT(bf16, tk::kBF16)

}  // extern "C"
