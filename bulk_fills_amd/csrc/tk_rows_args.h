// tk_rows_args.h -- arguments of the row operators' kernels, and the table of launches that
// each pair of types gives the entry points (tk_rows.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tk {

struct Drop {
  bool on;             // p > 0
  uint32_t hk;         // hash of the key
  uint32_t start;      // counter of element (0, 0)
  uint32_t threshold;  // kept where the word's low 23 bits reach ceil(p 2^23): u >= p, exactly
  float q;             // 1 - p
  float rq, rl;        // its reciprocal rounded down, and the rest
};

// Forward of the layer norm (x null: its input is `residual`) and of the fused operator.
struct FwdArgs {
  const void *x, *bias, *residual, *gamma, *beta;
  void *sum, *y;
  float *mean, *rstd;
  uint64_t rows, ldx, ldr, lds, ldy;
  uint32_t cols, waves;  // waves: of a row (kernels with a row to whole waves)
  float eps;
  bool params_f32, once;  // once: the call's reads go past the caches
  Drop drop;
};

// Backward of either (dx null: the layer norm alone, whose dx is `dresidual` here), and of
// dropout-add with a bias (dy is then of the residual stream's type, sum null).
struct BwdArgs {
  const void *dy, *dsum, *sum, *gamma;
  const float *mean, *rstd;
  void *dx, *dresidual;
  float *partial;  // lines of partial column sums: dgamma's, dbeta's, then dbias's
  void *sums[3];   // those gradients (null: not wanted), written by the kernel where `alone`
  float *stats;    // -rstd mean(g), -rstd mean(g h) of every row (wide rows)
  uint64_t rows, lddy, ldds, lds, lddx, lddr;
  uint32_t cols, waves, strip0;  // strip0: the launch's first strip of columns
  bool alone;                    // one line of sums: they are the gradients
  bool past;                     // the lines are written past the caches
  bool params_f32, once;  // once: the call's reads go past the caches
  Drop drop;
};

struct AddArgs {
  const void *x, *bias, *residual;
  void *y;
  uint64_t row0, ldx, ldr, ldy, cols64, bias_cols;
  uint32_t chunks, chunks_per_row, div_mul;
  int div_shift;
  bool flat;  // the call's matrices are one row of cols64 elements; a bias repeats in it
  bool params_f32, once;  // once: the call's reads go past the caches
  Drop drop;
};

// Floats from one line of partial sums to the next: a multiple of 128 bytes, so that no two
// work-groups write to one cache line (layer norm backward bf16 1000x1500: 10.1 us, packed 10.7).
constexpr uint64_t line_pitch(uint64_t cols) { return (cols + 31) & ~31ull; }

// How a backward call is cut: `lines` lines of partial sums.  Rows in registers (strips 0):
// `lanes` lanes to a row (64: row_waves whole waves), `waves` waves to a work-group.  Wide rows
// and dropout-add: `strips` strips of `lanes` lanes' columns.  `room`: lines that the workspace
// holds.
struct BwdPlan {
  int lanes, waves, row_waves;
  uint64_t lines, strips, room;
};

struct RowTable {
  int chunk;
  void (*norm_fwd)(const FwdArgs &, hipStream_t);
  void (*norm_bwd)(const BwdArgs &, const BwdPlan &, bool bias, hipStream_t);
  void (*add_bwd_sums)(const BwdArgs &, const BwdPlan &, hipStream_t);
  void (*add_fwd)(const AddArgs &, int chunk, hipStream_t);
  void (*add_bwd)(const AddArgs &, int chunk, hipStream_t);
};

// One for each pair of types (activations, residual stream).
RowTable rows_f32();
RowTable rows_f16();
RowTable rows_f16_r32();
RowTable rows_bf16();
RowTable rows_bf16_r32();

}  // namespace tk
