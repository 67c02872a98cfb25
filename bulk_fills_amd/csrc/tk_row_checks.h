// tk_row_checks.h -- what the entry points of the row operators and of those around them share on
// the host: argument checks, dropout's constants, workspaces.
#pragma once

#include <math.h>

#include "tk_internal.h"
#include "tk_rows_args.h"

namespace tk {

constexpr uint64_t kMaxDim = 1ull << 31, kMaxLd = 1ull << 31;
constexpr uint64_t kCachedReads = 96ull << 20;  // bytes a call may read through the caches (tk_rows.h)

struct Region {
  uintptr_t at;
  uint64_t rows, pitch, width;  // bytes
  int size;                     // element bytes
  bool out;
  int kind;  // 0: a vector; matrices of one kind may be the same (in place)
};

// Whether two arguments share bytes in a way a call may not have: an output matrix may be an
// input matrix of its kind; matrices of one pitch are told apart by their place within it.
inline bool clash(const Region &a, const Region &b) {
  if (!a.out && !b.out) return false;
  const uintptr_t ea = a.at + (a.rows - 1) * a.pitch + a.width, eb = b.at + (b.rows - 1) * b.pitch + b.width;
  if (ea <= b.at || eb <= a.at) return false;
  if (a.kind && b.kind) {
    if (a.kind == b.kind && a.at == b.at && a.size == b.size && (a.pitch == b.pitch || a.rows == 1)) return a.out && b.out;
    if (a.pitch == b.pitch && a.rows > 1) {
      const uint64_t d = b.at >= a.at ? (b.at - a.at) % a.pitch : (a.pitch - (a.at - b.at) % a.pitch) % a.pitch;
      return d < a.width || d + b.width > a.pitch;
    }
  }
  return true;
}

enum RowType { kF32, kF16, kBF16 };

struct Arguments {
  RowType type;
  uint64_t rows, cols;
  uint32_t flags;
  Region r[16];
  int n = 0;
  bool ok = true, range = true;
  int t() const { return type == kF32 ? 4 : 2; }
  int res() const { return flags & TK_RESIDUAL_F32 ? 4 : t(); }
  int par() const { return flags & TK_PARAMS_F32 ? 4 : t(); }
  void add(const void *p, uint64_t count, uint64_t ld, uint64_t width, int size, bool out, int kind) {
    if ((uintptr_t)p % size) ok = false;
    r[n++] = Region{(uintptr_t)p, count, ld * size, width * size, size, out, kind};
  }
  // A matrix of other sizes than the call's rows x cols.
  void matrix_of(const void *p, uint64_t count, uint64_t width, uint64_t ld, int size, bool out, bool needed, int kind) {
    if (!p) {
      ok = ok && !needed;
      return;
    }
    if (ld < width) ok = false;
    if (ld >= kMaxLd) range = false;
    else add(p, count, ld, width, size, out, kind);
  }
  void matrix(const void *p, uint64_t ld, int size, bool out, bool needed) {
    matrix_of(p, rows, cols, ld, size, out, needed, 1);
  }
  void vector(const void *p, uint64_t count, int size, bool out, bool needed) {
    if (!p) ok = ok && !needed;
    else add(p, 1, count, count, size, out, 0);
  }
  // Checks every pair; the caller has added all of a call's arguments.
  tk_status done() const {
    if (!ok) return TK_EINVAL;
    if (!range) return TK_ERANGE;
    for (int i = 0; i < n; ++i) {
      // a matrix must end below 2^57, above every address of a process: no sum of clash() wraps
      const unsigned __int128 end = (unsigned __int128)r[i].at + (unsigned __int128)(r[i].rows - 1) * r[i].pitch + r[i].width;
      if (end >> 57) return TK_ERANGE;
    }
    for (int i = 0; i < n; ++i)
      for (int j = i + 1; j < n; ++j)
        if (clash(r[i], r[j])) return TK_EINVAL;
    return TK_OK;
  }
};

inline tk_status check_scalars(uint64_t start, uint64_t rows, uint64_t cols, float p, float eps, uint32_t flags,
                               uint32_t allowed) {
  if (!(p >= 0.0f && p < 1.0f) || !(eps >= 0.0f && eps < INFINITY)) return TK_EINVAL;
  if (flags & ~allowed) return TK_EINVAL;
  if (rows >= kMaxDim || cols >= kMaxDim) return TK_ERANGE;
  if (p > 0.0f && (start > (1ull << 32) || rows * cols > (1ull << 32) - start)) return TK_ERANGE;
  return TK_OK;
}

inline bool params_f32(RowType t, uint32_t flags) { return t == kF32 || (flags & TK_PARAMS_F32); }

inline Drop drop_of(uint32_t key, uint64_t start, float p) {
  Drop d{};
  d.on = p > 0.0f;
  d.hk = host_lowbias32(key);
  d.start = (uint32_t)start;
  d.threshold = (uint32_t)ceilf(p * 0x1p23f);  // the product is exact
  d.q = 1.0f - p;
  const double r = 1.0 / (double)d.q;
  d.rq = (float)r;
  if (d.rq > r) d.rq = nextafterf(d.rq, 0.0f);
  // never 0 nor below, also where the reciprocal is a float: infinity times both is infinity
  d.rl = fmaxf((float)(r - d.rq), d.rq * 0x1p-48f);
  return d;
}

// Whether a workspace of `have` bytes serves.
inline bool serves(const void *workspace, uint64_t have, uint64_t need) {
  return need == 0 || (workspace && ((uintptr_t)workspace & 3u) == 0 && have >= need);
}

// Lines of partial column sums, one to a work-group: at most one work-group to a compute unit.
constexpr uint64_t kMaxLines = 256;

// Adds up `lines` lines of partial sums of up to three gradients (a, then b, then c; line_pitch(cols)
// floats a line) and writes them in the parameters' type; a null one's lines are there and skipped.
tk_status finish(RowType t, uint32_t flags, const float *partial, uint64_t lines, uint64_t cols, void *a, void *b, void *c,
                 hipStream_t stream);

}  // namespace tk
