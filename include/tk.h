/*
 * tk.h -- C ABI of libtk: counter-based random bulk fills into the device memory of one
 * AMD Instinct MI355X (gfx950).
 *
 * Contract (tandem-sycl, "Design", §Fills and §Normals): element k of a fill takes draw
 * i = start_draw + k, and its value is a pure function of (key, i).  A fill cut at any
 * element therefore equals the whole fill, and resuming a fill is a call with a larger
 * start_draw.  A start draw is an offset into the stream (tandem-cuda, "Performance",
 * §GPU: a row's start draw is a generator offset).
 *
 * Generator (Phobos stdlib, "Random numbers", §hash32 and §uniform): the lowbias32 hash,
 * word(key, c) = hash32(c ^ hash32(key)) for 32-bit key and counter.  Word c is the
 * stream's c-th 32-bit word; narrower draws are its little-endian parts and 64-bit draws
 * are the word pair (2i, 2i+1), low word first.  A fill whose counters would reach 2^32
 * is refused with TK_ERANGE instead of wrapping.
 *
 * Conventions for every call:
 *   - Pointers `out`, `x`, `y`, `mask` are device pointers owned by the caller; they must
 *     stay valid until the work enqueued on `stream` has finished.  The library never
 *     keeps them.  `out` must be aligned to its element size; any such alignment is
 *     accepted and fills at full speed (16-byte stores from the first 4 KiB boundary of
 *     `out`, the elements before it one at a time).
 *   - Calls are asynchronous and ordered on `stream` (NULL = the device's null stream)
 *     on the device current to the calling host thread.  Any host thread may call.
 *   - Arguments are checked before anything is enqueued; on any error nothing is
 *     enqueued.  n == 0 is TK_OK and enqueues nothing.  There is no CPU fallback.
 *   - TK_EHIP reports a HIP runtime failure; tk_last_hip_error() gives its code for the
 *     calling thread.
 *   - HIP graphs: a fill enqueues only kernel launches on `stream`, so it can be captured
 *     into a graph and replayed.  The first f64 normal fill on a device creates the
 *     library's per-device tables (an allocation and a copy), so run it once before
 *     capturing; alias tables are built and uploaded by tk_alias_create, outside any
 *     capture.  The test-hook modes of tk_debug_set_normal_f64_mode and the two-kernel
 *     path order fills by an event and are not meant for capture.
 */
#ifndef TK_H
#define TK_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum tk_status {
    TK_OK = 0,
    TK_EINVAL = 1, /* bad argument: NULL pointer, misaligned pointer, bad bound or p */
    TK_ERANGE = 2, /* draws beyond the 2^32-word counter space, or a bounded range whose
                      top does not fit the output type */
    TK_ENOMEM = 3, /* the library could not allocate its own device state */
    TK_EHIP = 4    /* a HIP runtime call failed */
} tk_status;

/* ---- Uniform fills ------------------------------------------------------------------
 * tandem-cuda, "Performance", §GPU table (fill_u8 ... fill_bool rows); narrow types write
 * fewer bytes of the same stream.
 *   u8:  draw i is byte i&3 of word i>>2          (i < 2^34)
 *   u16: draw i is half i&1 of word i>>1          (i < 2^33)
 *   u32: draw i is word i                         (i < 2^32)
 *   u64: draw i is word 2i | word 2i+1 << 32      (i < 2^31)
 *   f16_bits: binary16 encoding of (u16 draw & 0x7FF) * 2^-11, a uniform on [0, 1)
 *   f32: (word i & 0x7FFFFF) * 2^-23 (Phobos, §uniform), exactly
 *   f64: (u64 draw & (2^53 - 1)) * 2^-53, exactly
 *   bool: bit i&31 of word i>>5 as one byte 0 or 1 (tandem-sycl, "Design", §Fills: one
 *         byte per bit)                           (i < 2^37)                              */
tk_status tk_fill_u8(uint32_t key, uint64_t start_draw, uint64_t n, uint8_t *out, hipStream_t stream);
tk_status tk_fill_u16(uint32_t key, uint64_t start_draw, uint64_t n, uint16_t *out, hipStream_t stream);
tk_status tk_fill_u32(uint32_t key, uint64_t start_draw, uint64_t n, uint32_t *out, hipStream_t stream);
tk_status tk_fill_u64(uint32_t key, uint64_t start_draw, uint64_t n, uint64_t *out, hipStream_t stream);
tk_status tk_fill_f16_bits(uint32_t key, uint64_t start_draw, uint64_t n, uint16_t *out, hipStream_t stream);
tk_status tk_fill_f32(uint32_t key, uint64_t start_draw, uint64_t n, float *out, hipStream_t stream);
tk_status tk_fill_f64(uint32_t key, uint64_t start_draw, uint64_t n, double *out, hipStream_t stream);
tk_status tk_fill_bool(uint32_t key, uint64_t start_draw, uint64_t n, uint8_t *out, hipStream_t stream);

/* ---- Bounded integers ---------------------------------------------------------------
 * tandem-cuda, "Performance", §GPU (fill_u32_below, fill_u64_below, "with a low bound"
 * into int32_t / int64_t); perturbation-kernel, "Backends", §Why the GPU can be exact
 * (Lemire's multiply-shift with rejection).  Value = high half of x * bound for the
 * draw x, rejected while the low half is below (2^W - bound) mod bound; a rejected draw
 * continues on the per-index substream split(i) of sub(key, "BL32"/"BL64").
 * bound == 0 -> TK_EINVAL.  With `low`, values are low + [0, bound); a top
 * low + bound - 1 beyond the output type -> TK_ERANGE.
 *   u32_below, i32_below, i64_below32: one word per element (i < 2^32)
 *   u64_below, i64_below: one 64-bit draw per element (i < 2^31)                         */
tk_status tk_fill_u32_below(uint32_t key, uint64_t start_draw, uint64_t n, uint32_t bound,
                            uint32_t *out, hipStream_t stream);
tk_status tk_fill_u64_below(uint32_t key, uint64_t start_draw, uint64_t n, uint64_t bound,
                            uint64_t *out, hipStream_t stream);
tk_status tk_fill_i32_below(uint32_t key, uint64_t start_draw, uint64_t n, int32_t low,
                            uint32_t bound, int32_t *out, hipStream_t stream);
tk_status tk_fill_i64_below32(uint32_t key, uint64_t start_draw, uint64_t n, int64_t low,
                              uint32_t bound, int64_t *out, hipStream_t stream);
tk_status tk_fill_i64_below(uint32_t key, uint64_t start_draw, uint64_t n, int64_t low,
                            uint64_t bound, int64_t *out, hipStream_t stream);

/* ---- Normals ------------------------------------------------------------------------
 * f64 (tandem-sycl, "Design", §Normals): the 1024-layer equal-area ziggurat, one 64-bit
 * draw d per element: layer d & 1023, sign bit 10, u = (d >> 11) 2^-53; x = u X[layer] is
 * taken when below X[layer+1]; the ~0.43 % of draws that miss continue on the
 * per-index substream split(i) of sub(key, "NORM") (wedge test against exp(-x^2/2), or
 * the tail beyond r).  A table pass writes the fast-path values; the misses are finished
 * either by the same work-group after its stores or by a continuation pass over a miss
 * list (tk_debug_set_normal_f64_mode).  The 16 KiB layer table is constant per-device
 * library state; the miss lists and counts of the two-kernel path (and of counted test
 * fills) are per-device state ordered across streams by an event, while the default fused
 * fill keeps no mutable state and runs concurrently with fills on other streams.
 * i < 2^31.
 * f32 (tandem-sycl, "Design", §Normals; Phobos, §randn): Box-Muller pairs; draw i
 * belongs to pair c = i >> 1 built from the f32 uniforms at words 2c and 2c+1:
 * r = sqrt(-2 ln(1 - u1)), angle 2 pi t with t = u2 wrapped into [-1/2, 1/2); even i
 * takes r cos, odd i r sin.  i < 2^32.                                                   */
tk_status tk_fill_normal_f64(uint32_t key, uint64_t start_draw, uint64_t n, double *out, hipStream_t stream);
tk_status tk_fill_normal_f32(uint32_t key, uint64_t start_draw, uint64_t n, float *out, hipStream_t stream);

/* For callers that cannot allocate device memory (code under HIP graph capture, serving
 * loops, harnesses that forbid hipMalloc): tk_fill_normal_f64 computed by its two-kernel
 * path (table pass, then a continuation pass over the listed misses; the same values as
 * tk_fill_normal_f64) with no allocation of any kind.  The layer tables are compiled into
 * the library's device code, and the miss lists live in one static device array per device
 * (2.28 MiB, held from the first call on that device until the process ends); the call
 * enqueues three kernel launches on `stream` and nothing else.
 *   n: at most 2^24 elements per call, else TK_EINVAL (cut a longer fill into pieces on
 *      one stream: the pieces equal the whole fill).  Other arguments and errors as for
 *      tk_fill_normal_f64 (out 8-byte aligned, i < 2^31).
 *   Every call on a device uses that device's one array: calls that overlap in time on one
 *   device (other streams, other threads) race and give wrong values.  Order them, e.g. on
 *   one stream.  The array keeps the last call's contents; each call clears what must start
 *   at zero itself.                                                                      */
tk_status tk_fill_normal_f64_no_alloc(uint32_t key, uint64_t start_draw, uint64_t n, double *out,
                                      hipStream_t stream);

/* Normal variants (f32, i < 2^32 unless stated).
 * half_turn: tandem-sycl, "Design", §Normals shifts the Box-Muller angle by half a turn
 *   into [-pi, pi): the same pairs with angle 2 pi (u2 - 1/2), so both values are the
 *   negation of tk_fill_normal_f32's.
 * randn: Phobos, §randn, one normal per counter: element k is randn(key, start_draw + k),
 *   the cosine of Box-Muller pair start_draw + k (words 2c and 2c+1), i.e. element
 *   2 (start_draw + k) of tk_fill_normal_f32.  i < 2^31.                                 */
tk_status tk_fill_normal_f32_half_turn(uint32_t key, uint64_t start_draw, uint64_t n, float *out,
                                       hipStream_t stream);
tk_status tk_fill_randn_f32(uint32_t key, uint64_t start_draw, uint64_t n, float *out, hipStream_t stream);

/* ---- Exponentials ------------------------------------------------------------------
 * tandem-sycl, "Design", §Exponentials; tandem-cuda, "Performance", §GPU (the f32
 * exponential maps 1 - exp(-x) back to the draw's own 2^-24 grid point).  x = -ln(1 - u),
 * +0.0 at u = 0, by inversion of the draw's uniform:
 *   f64: u = (u64 draw & (2^53 - 1)) 2^-53; x from the library's table-driven f64
 *        logarithm (within 0.52 ulp of the exact value).                (i < 2^31)
 *   f32: u = (word i & 0xFFFFFF) 2^-24; x correctly rounded to f32 (the same logarithm
 *        rounded once, which is exact at every one of the 2^24 grid points).  (i < 2^32) */
tk_status tk_fill_exponential_f64(uint32_t key, uint64_t start_draw, uint64_t n, double *out, hipStream_t stream);
tk_status tk_fill_exponential_f32(uint32_t key, uint64_t start_draw, uint64_t n, float *out, hipStream_t stream);

/* ---- Fused dropout ------------------------------------------------------------------
 * Phobos, §dropout: y[k] = uniform(key, start_draw + k) >= p ? x[k] / (1 - p) : +0.0, with
 * 1 - p and the quotient rounded as f32 operations (a true division).  p must lie in
 * [0, 1), else TK_EINVAL.  x and y are n floats; they may be the same buffer (in place)
 * but must not otherwise overlap.  mask (nullable) receives one byte per element, 1 for
 * kept.  i < 2^32.                                                                       */
tk_status tk_dropout_f32(uint32_t key, uint64_t start_draw, uint64_t n, float p, const float *x,
                         float *y, uint8_t *mask, hipStream_t stream);

/* Dropout backward by redrawing (Phobos, §Random numbers: the same seed and counter give
 * the same number, so a backward pass redraws its forward pass's mask instead of storing
 * it): dx[k] = keep(k) ? dy[k] / (1 - p) : +0.0, where keep(k) is the decision of
 * tk_dropout_f32 for the same key, start_draw + k and p.  The same computation as the
 * forward call applied to dy with no mask output; same checks (dy and dx may be the same
 * buffer, no other overlap).  i < 2^32.                                                 */
tk_status tk_dropout_backward_f32(uint32_t key, uint64_t start_draw, uint64_t n, float p, const float *dy,
                                  float *dx, hipStream_t stream);

/* ---- Row operators: dropout-add and layer norm ---------------------------------------
 * The dropout of a transformer block at its place: after a bias, before the residual, and
 * with the layer norm that reads the sum.  Every operator works on a rows x cols matrix of
 * float (_f32), binary16 (_f16) or bfloat16 (_bf16) elements and computes in float, rounding
 * each output once.  With z = x + bias and drop(v) at (r, c) = v / (1 - p) where the f32
 * uniform of word start_draw + r * cols + c is at least p, else +0.0 (Phobos, §dropout: the
 * decision of tk_dropout_f32 with the flat index as its counter, so a fill cut at any row
 * equals the whole and the backward pass redraws the mask):
 *   tk_dropout_add             y = residual + drop(z)
 *     _backward                dx = drop(dy);  dbias = column sums of dx.  (residual's
 *                              gradient is dy itself.)
 *   tk_layer_norm              y = h gamma + beta, h = (x - mean) rstd, with the row's mean and
 *                              rstd = 1 / sqrt(variance + eps), variance = mean of (x - mean)^2
 *     _backward                g = dy gamma:  dx = rstd (g - mean(g) - h mean(g h)),
 *                              dgamma = column sums of dy h, dbeta = column sums of dy
 *   tk_dropout_add_layer_norm  sum = residual + drop(z);  y = layer norm of that sum (before
 *                              sum's own rounding)
 *     _backward                dresidual = dsum + dx of the layer norm at `sum`;
 *                              dx = drop(dresidual);  dbias = column sums of dx;  dgamma, dbeta
 * The quotient is the IEEE division in the _f32 operators (as in tk_dropout_f32).  The 16-bit
 * ones multiply by 1 / (1 - p), held to 2^-46, and round once to float: the quotient's float
 * but next to the middle of two.  p == 0
 * keeps every element and takes no draws (no limit on the counters then).
 *   flags: TK_RESIDUAL_F32  the residual stream is float: residual, dropout-add's y and dy,
 *                           sum, dsum, dresidual, and tk_layer_norm's x and dx
 *          TK_PARAMS_F32    bias, gamma, beta and their gradients are float
 *          (both change nothing for _f32; other bits: TK_EINVAL)
 *   Nullable: bias, residual, beta and gamma (0, 0, 0 and 1 in their place), dsum (0), and the
 *          outputs sum, mean, rstd, dgamma, dbeta, dbias and the fused backward's dresidual.
 *   ld*:   elements from a matrix's row to its next, at least cols.  Elements between the rows
 *          are neither read nor written.  mean and rstd are `rows` floats; the backward takes
 *          those that the forward wrote.  Any element-aligned address is accepted.
 *   In place: an output matrix may be an input matrix (same address, ld and element type).
 *          Otherwise no output may share bytes with any other argument; slices of one buffer
 *          with one row pitch are told apart exactly, other matrices by their whole extent.
 *   p must lie in [0, 1) and eps be finite and >= 0, else TK_EINVAL.  rows and cols are below
 *          2^31 and so is ld, else TK_ERANGE; start_draw + rows * cols <= 2^32 where
 *          p > 0, else TK_ERANGE.  rows == 0 or cols == 0 is TK_OK: the forward calls and dx
 *          have nothing to write, gradients over rows == 0 are written as zeros.
 *   workspace: the backward calls that give dgamma, dbeta or dbias, and those of the layer
 *          norms at more than 8192 columns, need device memory of at least the size that
 *          tk_backward_workspace_bytes names (64-bit count in *bytes; TK_ERANGE as above),
 *          4-byte aligned, else TK_EINVAL (a size of 0: none is needed, as where one work-group
 *          takes all rows).  The size never falls as rows grow, so one for the most rows serves
 *          all.  It holds nothing between calls; calls that may overlap in time (other streams,
 *          graphs replayed together) need one each.
 * Far from zero: the forward's y holds h to float also where the mean is many times the row's
 *          spread.  The backward's h is made from the mean as a float, so it is off by up to
 *          2^-24 |mean| rstd there.
 * NaN and infinity follow the formulas; a dropped element is +0.0 whatever it was.  Column
 * sums are taken in a fixed order: equal arguments give equal bits, run after run.          */
#define TK_RESIDUAL_F32 1u
#define TK_PARAMS_F32 2u
tk_status tk_backward_workspace_bytes(uint64_t rows, uint64_t cols, uint64_t *bytes);

tk_status tk_dropout_add_f32(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p, uint32_t flags,
        const void *x, uint64_t ldx, const void *bias, const void *residual, uint64_t ldr, void *y, uint64_t ldy,
        hipStream_t stream);
tk_status tk_dropout_add_backward_f32(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p,
        uint32_t flags, const void *dy, uint64_t lddy, void *dx, uint64_t lddx, void *dbias, void *workspace,
        uint64_t workspace_bytes, hipStream_t stream);
tk_status tk_layer_norm_f32(uint64_t rows, uint64_t cols, float eps, uint32_t flags, const void *x, uint64_t ldx,
        const void *gamma, const void *beta, void *y, uint64_t ldy, float *mean, float *rstd, hipStream_t stream);
tk_status tk_layer_norm_backward_f32(uint64_t rows, uint64_t cols, uint32_t flags, const void *dy, uint64_t lddy,
        const void *x, uint64_t ldx, const void *gamma, const float *mean, const float *rstd, void *dx, uint64_t lddx,
        void *dgamma, void *dbeta, void *workspace, uint64_t workspace_bytes, hipStream_t stream);
tk_status tk_dropout_add_layer_norm_f32(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p,
        float eps, uint32_t flags, const void *x, uint64_t ldx, const void *bias, const void *residual, uint64_t ldr,
        const void *gamma, const void *beta, void *sum, uint64_t lds, void *y, uint64_t ldy, float *mean, float *rstd,
        hipStream_t stream);
tk_status tk_dropout_add_layer_norm_backward_f32(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols,
        float p, uint32_t flags, const void *dy, uint64_t lddy, const void *dsum, uint64_t ldds, const void *sum,
        uint64_t lds, const void *gamma, const float *mean, const float *rstd, void *dx, uint64_t lddx,
        void *dresidual, uint64_t lddr, void *dgamma, void *dbeta, void *dbias, void *workspace,
        uint64_t workspace_bytes, hipStream_t stream);

tk_status tk_dropout_add_f16(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p, uint32_t flags,
        const void *x, uint64_t ldx, const void *bias, const void *residual, uint64_t ldr, void *y, uint64_t ldy,
        hipStream_t stream);
tk_status tk_dropout_add_backward_f16(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p,
        uint32_t flags, const void *dy, uint64_t lddy, void *dx, uint64_t lddx, void *dbias, void *workspace,
        uint64_t workspace_bytes, hipStream_t stream);
tk_status tk_layer_norm_f16(uint64_t rows, uint64_t cols, float eps, uint32_t flags, const void *x, uint64_t ldx,
        const void *gamma, const void *beta, void *y, uint64_t ldy, float *mean, float *rstd, hipStream_t stream);
tk_status tk_layer_norm_backward_f16(uint64_t rows, uint64_t cols, uint32_t flags, const void *dy, uint64_t lddy,
        const void *x, uint64_t ldx, const void *gamma, const float *mean, const float *rstd, void *dx, uint64_t lddx,
        void *dgamma, void *dbeta, void *workspace, uint64_t workspace_bytes, hipStream_t stream);
tk_status tk_dropout_add_layer_norm_f16(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p,
        float eps, uint32_t flags, const void *x, uint64_t ldx, const void *bias, const void *residual, uint64_t ldr,
        const void *gamma, const void *beta, void *sum, uint64_t lds, void *y, uint64_t ldy, float *mean, float *rstd,
        hipStream_t stream);
tk_status tk_dropout_add_layer_norm_backward_f16(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols,
        float p, uint32_t flags, const void *dy, uint64_t lddy, const void *dsum, uint64_t ldds, const void *sum,
        uint64_t lds, const void *gamma, const float *mean, const float *rstd, void *dx, uint64_t lddx,
        void *dresidual, uint64_t lddr, void *dgamma, void *dbeta, void *dbias, void *workspace,
        uint64_t workspace_bytes, hipStream_t stream);

tk_status tk_dropout_add_bf16(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p, uint32_t flags,
        const void *x, uint64_t ldx, const void *bias, const void *residual, uint64_t ldr, void *y, uint64_t ldy,
        hipStream_t stream);
tk_status tk_dropout_add_backward_bf16(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p,
        uint32_t flags, const void *dy, uint64_t lddy, void *dx, uint64_t lddx, void *dbias, void *workspace,
        uint64_t workspace_bytes, hipStream_t stream);
tk_status tk_layer_norm_bf16(uint64_t rows, uint64_t cols, float eps, uint32_t flags, const void *x, uint64_t ldx,
        const void *gamma, const void *beta, void *y, uint64_t ldy, float *mean, float *rstd, hipStream_t stream);
tk_status tk_layer_norm_backward_bf16(uint64_t rows, uint64_t cols, uint32_t flags, const void *dy, uint64_t lddy,
        const void *x, uint64_t ldx, const void *gamma, const float *mean, const float *rstd, void *dx, uint64_t lddx,
        void *dgamma, void *dbeta, void *workspace, uint64_t workspace_bytes, hipStream_t stream);
tk_status tk_dropout_add_layer_norm_bf16(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p,
        float eps, uint32_t flags, const void *x, uint64_t ldx, const void *bias, const void *residual, uint64_t ldr,
        const void *gamma, const void *beta, void *sum, uint64_t lds, void *y, uint64_t ldy, float *mean, float *rstd,
        hipStream_t stream);
tk_status tk_dropout_add_layer_norm_backward_bf16(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols,
        float p, uint32_t flags, const void *dy, uint64_t lddy, const void *dsum, uint64_t ldds, const void *sum,
        uint64_t lds, const void *gamma, const float *mean, const float *rstd, void *dx, uint64_t lddx,
        void *dresidual, uint64_t lddr, void *dgamma, void *dbeta, void *dbias, void *workspace,
        uint64_t workspace_bytes, hipStream_t stream);

/* ---- Embedding lookup ----------------------------------------------------------------
 * The rows' way into a model, and the table's gradient, with the dropout that follows the lookup.
 * Types, flags, strides, rounding and drop() are the row operators'; the counter of an element is
 * start_draw + r * cols + c:
 *   tk_embedding     y[r] = drop(scale * table[ids[r]])
 *     _backward      dtable[v] = scale * (sum of drop(dy[r]) over the rows r with ids[r] = v)
 * ids are `rows` int32 numbers, or int64 with TK_INDEX_I64.  table and dtable are vocab x cols.  A row
 * whose id is no row of the table (below 0, as padding often is, or vocab and above) gives a y of
 * +0.0 and goes into no gradient; its dy is not read.
 *   flags: TK_RESIDUAL_F32  y and dy are float       TK_PARAMS_F32  table and dtable are float
 *          TK_INDEX_I64     ids are int64
 *          TK_ACCUMULATE    (backward) scale * sum, rounded to a float, is added to what dtable holds, as
 *                           floats, and that rounded to dtable's type; rows of it whose token does not
 *                           occur are neither read nor written.  Without it every row is written, with
 *                           zeros where its token does not occur.
 * The gradient's sums are float, in an order that the arguments fix: equal arguments give equal bits.
 * Nothing is updated concurrently: the rows, sorted by token, are summed in pieces of 8 to 64, and the pieces of
 * one token are then added one after the other.  So a token that has most of a call's rows makes it longer,
 * the more rows and the narrower they are: bf16, vocabulary 32768, all rows one token's 250 us for 32768 x 64
 * (evenly spread 29), 177 for 32768 x 512 (36), 111 for 16384 x 4096 (98).  A row of padding is best given
 * an id that is no row of the table.
 *   scale must be finite, else TK_EINVAL; rows, cols, vocab and the lds are below 2^31, else TK_ERANGE.
 *   rows == 0 or cols == 0 is TK_OK, as is vocab == 0 (y is then zeros; the table may be NULL);
 *   a gradient over rows == 0 is zeros, or with TK_ACCUMULATE stays as it is.
 *   No output may share bytes with any other argument.
 *   workspace (backward): at least the bytes that tk_embedding_workspace_bytes names, 4-byte aligned;
 *   as for the row operators it holds nothing between calls, one for the most rows serves fewer, and
 *   calls that may overlap in time need one each.                                              */
#define TK_INDEX_I64 8u
#define TK_ACCUMULATE 16u
tk_status tk_embedding_workspace_bytes(uint64_t rows, uint64_t cols, uint64_t vocab, uint64_t *bytes);

tk_status tk_embedding_f32(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p, float scale,
        uint32_t flags, uint64_t vocab, const void *ids, const void *table, uint64_t ldt, void *y, uint64_t ldy,
        hipStream_t stream);
tk_status tk_embedding_backward_f32(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p, float scale,
        uint32_t flags, uint64_t vocab, const void *ids, const void *dy, uint64_t lddy, void *dtable, uint64_t lddt,
        void *workspace, uint64_t workspace_bytes, hipStream_t stream);

tk_status tk_embedding_f16(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p, float scale,
        uint32_t flags, uint64_t vocab, const void *ids, const void *table, uint64_t ldt, void *y, uint64_t ldy,
        hipStream_t stream);
tk_status tk_embedding_backward_f16(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p, float scale,
        uint32_t flags, uint64_t vocab, const void *ids, const void *dy, uint64_t lddy, void *dtable, uint64_t lddt,
        void *workspace, uint64_t workspace_bytes, hipStream_t stream);

tk_status tk_embedding_bf16(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p, float scale,
        uint32_t flags, uint64_t vocab, const void *ids, const void *table, uint64_t ldt, void *y, uint64_t ldy,
        hipStream_t stream);
tk_status tk_embedding_backward_bf16(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, float p, float scale,
        uint32_t flags, uint64_t vocab, const void *ids, const void *dy, uint64_t lddy, void *dtable, uint64_t lddt,
        void *workspace, uint64_t workspace_bytes, hipStream_t stream);

/* ---- Norms of queries and keys for each head, with the position rotation -------------
 * A row is a token: heads_q query heads and heads_k key heads of `dim` elements each, one after the
 * other in q's row and in k's (slices of one projection's output, by their ld, as well as matrices of
 * their own).  For each head x:
 *   n = x rstd gamma, rstd = 1 / sqrt(mean(x^2) + eps), with gamma_q or gamma_k of dim elements;
 *   the first `rotary` elements of n turn in pairs (a, b), i < rotary / 2:
 *     (a cos - b sin, b cos + a sin),  cos = cosines[pos][i], sin = sines[pos][i],
 *   where a and b are elements i and rotary / 2 + i, or with TK_INTERLEAVED 2 i and 2 i + 1; the rest
 *   of the head stays as it is.
 * pos is positions[r], int32 or with TK_INDEX_I64 int64 (NULL: r).  cosines and sines are table_rows x
 * (rotary / 2) contiguous floats that the caller makes once.  A row whose position is not in
 * [0, table_rows), padding for instance, is normed and does not turn.
 *   _backward: g = dy turned back, h = x rstd: dgamma = sums of g h over rows and heads,
 *              dx = rstd (g gamma - h mean(g gamma h)); the statistics are made anew from x.
 * All matrices are of the operator's type; sums and angles are float, outputs are rounded once.
 * The sum of a head's squares is a float as well: a head where it passes float's range (2^128: elements of
 * 2^60 and more, as the lowest value of float or bfloat16 is) comes out as zeros, and so do its gradients; an
 * element below 2^-75 adds nothing to it, so that a head of such alone gives infinities or NaN where eps is 0.
 * NaN and infinity follow the formulas and stay in their head.
 *   flags: TK_PARAMS_F32 (gammas and their gradients are float), TK_INDEX_I64, TK_INTERLEAVED.
 *   Nullable: gammas (1), positions, dgammas, q's or k's arguments where their number of heads is 0,
 *          and the tables where rotary or table_rows is 0.
 *   In place: yq may be q and yk k; dq may be q or dyq, dk k or dyk (same address and ld).  No other
 *          output may share bytes with any other argument.
 *   rotary must be even and at most dim, else TK_EINVAL; dim is at most 512, and rows, a row's
 *   elements, the heads of all rows, table_rows and the lds are below 2^31, else TK_ERANGE.  rows == 0, dim == 0 or no head at
 *   all is TK_OK with nothing to write but gradients of gammas, which are zeros.
 *   workspace (backward with dgamma_q or dgamma_k): at least the bytes that
 *   tk_head_norm_workspace_bytes names, 4-byte aligned; rules as above.                        */
#define TK_INTERLEAVED 32u
tk_status tk_head_norm_workspace_bytes(uint64_t rows, uint64_t heads_q, uint64_t heads_k, uint64_t dim, uint64_t *bytes);

tk_status tk_head_norm_rotate_f32(uint64_t rows, uint64_t heads_q, uint64_t heads_k, uint64_t dim, uint64_t rotary,
        float eps, uint32_t flags, const void *q, uint64_t ldq, const void *k, uint64_t ldk, const void *gamma_q,
        const void *gamma_k, const void *positions, uint64_t table_rows, const float *cosines, const float *sines,
        void *yq, uint64_t ldyq, void *yk, uint64_t ldyk, hipStream_t stream);
tk_status tk_head_norm_rotate_backward_f32(uint64_t rows, uint64_t heads_q, uint64_t heads_k, uint64_t dim,
        uint64_t rotary, float eps, uint32_t flags, const void *dyq, uint64_t lddyq, const void *dyk, uint64_t lddyk,
        const void *q, uint64_t ldq, const void *k, uint64_t ldk, const void *gamma_q, const void *gamma_k,
        const void *positions, uint64_t table_rows, const float *cosines, const float *sines, void *dq, uint64_t lddq,
        void *dk, uint64_t lddk, void *dgamma_q, void *dgamma_k, void *workspace, uint64_t workspace_bytes,
        hipStream_t stream);

tk_status tk_head_norm_rotate_f16(uint64_t rows, uint64_t heads_q, uint64_t heads_k, uint64_t dim, uint64_t rotary,
        float eps, uint32_t flags, const void *q, uint64_t ldq, const void *k, uint64_t ldk, const void *gamma_q,
        const void *gamma_k, const void *positions, uint64_t table_rows, const float *cosines, const float *sines,
        void *yq, uint64_t ldyq, void *yk, uint64_t ldyk, hipStream_t stream);
tk_status tk_head_norm_rotate_backward_f16(uint64_t rows, uint64_t heads_q, uint64_t heads_k, uint64_t dim,
        uint64_t rotary, float eps, uint32_t flags, const void *dyq, uint64_t lddyq, const void *dyk, uint64_t lddyk,
        const void *q, uint64_t ldq, const void *k, uint64_t ldk, const void *gamma_q, const void *gamma_k,
        const void *positions, uint64_t table_rows, const float *cosines, const float *sines, void *dq, uint64_t lddq,
        void *dk, uint64_t lddk, void *dgamma_q, void *dgamma_k, void *workspace, uint64_t workspace_bytes,
        hipStream_t stream);

tk_status tk_head_norm_rotate_bf16(uint64_t rows, uint64_t heads_q, uint64_t heads_k, uint64_t dim, uint64_t rotary,
        float eps, uint32_t flags, const void *q, uint64_t ldq, const void *k, uint64_t ldk, const void *gamma_q,
        const void *gamma_k, const void *positions, uint64_t table_rows, const float *cosines, const float *sines,
        void *yq, uint64_t ldyq, void *yk, uint64_t ldyk, hipStream_t stream);
tk_status tk_head_norm_rotate_backward_bf16(uint64_t rows, uint64_t heads_q, uint64_t heads_k, uint64_t dim,
        uint64_t rotary, float eps, uint32_t flags, const void *dyq, uint64_t lddyq, const void *dyk, uint64_t lddyk,
        const void *q, uint64_t ldq, const void *k, uint64_t ldk, const void *gamma_q, const void *gamma_k,
        const void *positions, uint64_t table_rows, const float *cosines, const float *sines, void *dq, uint64_t lddq,
        void *dk, uint64_t lddk, void *dgamma_q, void *dgamma_k, void *workspace, uint64_t workspace_bytes,
        hipStream_t stream);

/* ---- Activation checkpoints in 8 bits --------------------------------------------------
 * What the backward pass needs of the forward one, kept in a byte an element: a row's columns in blocks
 * of 128, each with a float scale.  With m = the block's largest |x|:
 *   scale = m / 127, inverse = 127 / m and t = |x| inverse, each rounded to float;
 *   code = sign(x) min(127, floor(t) + (u < t - floor(t))),  u = the f32 uniform of word
 *   start_draw + r * cols + c (Phobos, uniform): rounded up with the chance of its fraction, so that
 *   code * scale is x on average.  The comparison is exact: equal arguments give equal codes on
 *   any device.
 * A block whose m is below 2^-100 is kept as zeros (scale 0); one that holds an infinity or a NaN comes
 * back as NaN throughout (scale NaN, codes 0).  Where values are made from codes, a scale counts as at most
 * float's largest / 127 rounded down: that of a block that holds float's largest is one unit of its last
 * place above, and 127 times it would be infinite.
 *   tk_checkpoint          x (float with TK_RESIDUAL_F32, the only flag) to codes, rows x cols bytes
 *                          `ldc` apart, and scales, rows x ceil(cols / 128) contiguous floats
 *   tk_checkpoint_restore  y = code * scale, a float's product, rounded to y's type
 *   tk_layer_norm_backward_checkpoint, tk_dropout_add_layer_norm_backward_checkpoint
 *                          the backward passes of the row operators with the checkpoint in place of x or
 *                          sum, its values float; mean and rstd are the forward's
 * Overlaps, limits and the backward passes' workspace (tk_backward_workspace_bytes) are the row
 * operators'; codes and scales are in no place of another argument.  start_draw + rows * cols <= 2^32
 * (tk_checkpoint always), else TK_ERANGE.                                                      */
tk_status tk_checkpoint_f32(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, uint32_t flags, const void *x,
        uint64_t ldx, int8_t *codes, uint64_t ldc, float *scales, hipStream_t stream);
tk_status tk_checkpoint_restore_f32(uint64_t rows, uint64_t cols, uint32_t flags, const int8_t *codes, uint64_t ldc,
        const float *scales, void *y, uint64_t ldy, hipStream_t stream);
tk_status tk_layer_norm_backward_checkpoint_f32(uint64_t rows, uint64_t cols, uint32_t flags, const void *dy,
        uint64_t lddy, const int8_t *codes, uint64_t ldc, const float *scales, const void *gamma, const float *mean,
        const float *rstd, void *dx, uint64_t lddx, void *dgamma, void *dbeta, void *workspace,
        uint64_t workspace_bytes, hipStream_t stream);
tk_status tk_dropout_add_layer_norm_backward_checkpoint_f32(uint32_t key, uint64_t start_draw, uint64_t rows,
        uint64_t cols, float p, uint32_t flags, const void *dy, uint64_t lddy, const void *dsum, uint64_t ldds,
        const int8_t *codes, uint64_t ldc, const float *scales, const void *gamma, const float *mean,
        const float *rstd, void *dx, uint64_t lddx, void *dresidual, uint64_t lddr, void *dgamma, void *dbeta,
        void *dbias, void *workspace, uint64_t workspace_bytes, hipStream_t stream);

tk_status tk_checkpoint_f16(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, uint32_t flags, const void *x,
        uint64_t ldx, int8_t *codes, uint64_t ldc, float *scales, hipStream_t stream);
tk_status tk_checkpoint_restore_f16(uint64_t rows, uint64_t cols, uint32_t flags, const int8_t *codes, uint64_t ldc,
        const float *scales, void *y, uint64_t ldy, hipStream_t stream);
tk_status tk_layer_norm_backward_checkpoint_f16(uint64_t rows, uint64_t cols, uint32_t flags, const void *dy,
        uint64_t lddy, const int8_t *codes, uint64_t ldc, const float *scales, const void *gamma, const float *mean,
        const float *rstd, void *dx, uint64_t lddx, void *dgamma, void *dbeta, void *workspace,
        uint64_t workspace_bytes, hipStream_t stream);
tk_status tk_dropout_add_layer_norm_backward_checkpoint_f16(uint32_t key, uint64_t start_draw, uint64_t rows,
        uint64_t cols, float p, uint32_t flags, const void *dy, uint64_t lddy, const void *dsum, uint64_t ldds,
        const int8_t *codes, uint64_t ldc, const float *scales, const void *gamma, const float *mean,
        const float *rstd, void *dx, uint64_t lddx, void *dresidual, uint64_t lddr, void *dgamma, void *dbeta,
        void *dbias, void *workspace, uint64_t workspace_bytes, hipStream_t stream);

tk_status tk_checkpoint_bf16(uint32_t key, uint64_t start_draw, uint64_t rows, uint64_t cols, uint32_t flags, const void *x,
        uint64_t ldx, int8_t *codes, uint64_t ldc, float *scales, hipStream_t stream);
tk_status tk_checkpoint_restore_bf16(uint64_t rows, uint64_t cols, uint32_t flags, const int8_t *codes, uint64_t ldc,
        const float *scales, void *y, uint64_t ldy, hipStream_t stream);
tk_status tk_layer_norm_backward_checkpoint_bf16(uint64_t rows, uint64_t cols, uint32_t flags, const void *dy,
        uint64_t lddy, const int8_t *codes, uint64_t ldc, const float *scales, const void *gamma, const float *mean,
        const float *rstd, void *dx, uint64_t lddx, void *dgamma, void *dbeta, void *workspace,
        uint64_t workspace_bytes, hipStream_t stream);
tk_status tk_dropout_add_layer_norm_backward_checkpoint_bf16(uint32_t key, uint64_t start_draw, uint64_t rows,
        uint64_t cols, float p, uint32_t flags, const void *dy, uint64_t lddy, const void *dsum, uint64_t ldds,
        const int8_t *codes, uint64_t ldc, const float *scales, const void *gamma, const float *mean,
        const float *rstd, void *dx, uint64_t lddx, void *dresidual, uint64_t lddr, void *dgamma, void *dbeta,
        void *dbias, void *workspace, uint64_t workspace_bytes, hipStream_t stream);

/* ---- Weighted choice through an alias table -----------------------------------------
 * tandem-sycl, "Design", §Fills: the choice fill maps each 64-bit draw through an alias
 * table.  tk_alias_create builds the table on the host from n >= 1 finite, non-negative
 * host weights with a positive sum (integer Vose construction: index j owns an integer
 * share of n * 2^32, the rounding remainder going to the largest weight) and uploads it
 * to the current device; it is synchronous and owns its device memory until
 * tk_alias_destroy.  The fill maps draw d to column c = (hi32(d) * n) >> 32 and coin
 * lo32(d): out = coin < q[c] ? c : alias[c].  The table must outlive the stream work that
 * reads it and be used on the device it was created on.  i < 2^31.                       */
typedef struct tk_alias tk_alias;
tk_status tk_alias_create(const double *weights, uint32_t n, tk_alias **table);
tk_status tk_alias_destroy(tk_alias *table);
uint32_t tk_alias_size(const tk_alias *table);
/* The host construction tk_alias_create uploads, alone: writes n entries of q and alias
 * to host arrays.  Touches no device. */
tk_status tk_alias_build_host(const double *weights, uint32_t n, uint32_t *q, uint32_t *alias);
/* Copies the table to host arrays of tk_alias_size() entries each. */
tk_status tk_alias_export(const tk_alias *table, uint32_t *q, uint32_t *alias);
tk_status tk_fill_choice_u32(uint32_t key, uint64_t start_draw, uint64_t n, const tk_alias *table,
                             uint32_t *out, hipStream_t stream);

/* ---- Philox4x32-10 word source ------------------------------------------------------
 * The counter-based generator of the cuRAND comparison column (tandem-cuda,
 * "Performance", §GPU); Salmon et al., SC'11.  64-bit key (lo, hi); word w is lane w & 3
 * of the block with counter (lo32(w >> 2), hi32(w >> 2), 0, 0).  Same draw layout and
 * float transforms as the lowbias32 fills; the counter space is 64-bit.                  */
tk_status tk_philox_fill_u32(uint64_t key, uint64_t start_draw, uint64_t n, uint32_t *out, hipStream_t stream);
tk_status tk_philox_fill_u64(uint64_t key, uint64_t start_draw, uint64_t n, uint64_t *out, hipStream_t stream);
tk_status tk_philox_fill_f32(uint64_t key, uint64_t start_draw, uint64_t n, float *out, hipStream_t stream);
tk_status tk_philox_fill_f64(uint64_t key, uint64_t start_draw, uint64_t n, double *out, hipStream_t stream);

/* Philox variants of the bounded, choice and normal fills: the same definitions as the
 * lowbias32 fills above, over Philox words (u32 draw i = word i; 64-bit draw i = words 2i
 * and 2i+1).  A draw that is rejected (Lemire) or misses the ziggurat's fast path continues
 * on its Philox substream: word j of draw i's substream for purpose P ("BL32", "BL64",
 * "NORM") is lane j & 3 of the block with counter (lo32 i, hi32 i, P, j >> 2), disjoint
 * from the primary blocks.  Limits: u32_below and normal_f32 i < 2^64, u64_below, choice
 * and normal_f64 i < 2^63; normal_f64 takes n < 2^32 per call (cut a longer fill: the
 * pieces equal the whole).  bound == 0 is TK_EINVAL.  The choice table must be on the
 * current device, as for tk_fill_choice_u32.                                            */
tk_status tk_philox_fill_u32_below(uint64_t key, uint64_t start_draw, uint64_t n, uint32_t bound, uint32_t *out,
                                   hipStream_t stream);
tk_status tk_philox_fill_u64_below(uint64_t key, uint64_t start_draw, uint64_t n, uint64_t bound, uint64_t *out,
                                   hipStream_t stream);
tk_status tk_philox_fill_choice_u32(uint64_t key, uint64_t start_draw, uint64_t n, const tk_alias *table,
                                    uint32_t *out, hipStream_t stream);
tk_status tk_philox_fill_normal_f32(uint64_t key, uint64_t start_draw, uint64_t n, float *out, hipStream_t stream);
tk_status tk_philox_fill_normal_f64(uint64_t key, uint64_t start_draw, uint64_t n, double *out, hipStream_t stream);

/* ---- Store ceiling ------------------------------------------------------------------
 * The store path alone: out[k] = value for k < n, written with exactly the streaming
 * fills' geometry, grid and 16-byte stores and no generator.  The rate at which the device
 * takes this kernel's stores is the measured ceiling the fills are reported against (the
 * pages' fills run at ~95 % of their GPU's bandwidth: tandem-cuda, "Performance", §GPU and
 * the notes under its table).  out must be 4-byte aligned; n * 4 must fit 64 bits, else
 * TK_ERANGE.                                                                            */
tk_status tk_fill_constant_u32(uint32_t value, uint64_t n, uint32_t *out, hipStream_t stream);

/* ---- Status and introspection -------------------------------------------------------*/
const char *tk_status_string(tk_status status);
/* The hipError_t of the last TK_EHIP returned to the calling thread (0 if none). */
int tk_last_hip_error(void);
/* Copies the 1024-layer table the kernels use: x and f of 1025 doubles each (host). */
tk_status tk_ziggurat_table(double *x, double *f);
/* Test hook for the f64 normal's miss lists, applied from the next tk_fill_normal_f64 on
 * every device: each table-pass work-group keeps at most `per_group` misses (1..16) in its
 * queue.  In the two-kernel mode the rest go to an overflow list of `overflow` entries,
 * and when that overflows too the continuation pass walks the whole fill; in the fused
 * mode a group with more misses walks its own elements again.  0 restores the defaults
 * (16 per 4 KiB tile, 65536 overflow entries).  Lets tests force every fallback. */
tk_status tk_debug_set_miss_capacity(uint32_t per_group, uint64_t overflow);
/* Test hook: how tk_fill_normal_f64 finishes its misses, from the next call on every
 * device: 1 = the two-kernel path (table pass, then a continuation pass over the listed
 * misses), 2 = fused (each table-pass work-group finishes its own misses after its
 * stores), 0 = the library default.  Both give identical results. */
tk_status tk_debug_set_normal_f64_mode(uint32_t mode);
/* Test hook: waits for the current device's last tk_fill_normal_f64 and returns how many
 * of its draws missed the fast path (synchronous).  The counts are kept only while a mode
 * is chosen with tk_debug_set_normal_f64_mode (1 or 2), or when the library default is
 * the two-kernel path; after a fill in the default fused mode, which keeps no per-device
 * state and is not ordered against fills on other streams, it returns TK_EINVAL. */
tk_status tk_debug_last_miss_count(uint64_t *count);
/* Test hook: of the library's next device allocations (a device's ziggurat tables on its
 * first f64 normal fill, the two-kernel path's miss lists as they grow, alias tables), the
 * first `skip` proceed and the `count` after them fail as if device memory were exhausted,
 * without calling HIP.  The call that needed the memory returns TK_ENOMEM, enqueues
 * nothing and holds no more device memory than before it (a first fill releases the
 * tables it created; a failed growth releases all the miss lists); a later call allocates
 * again.  count = 0 cancels.  Process-wide, for every device and thread.  A real
 * allocation failure takes the same path.  The environment variable TK_DEBUG_FAIL_ALLOC=<n>
 * makes the process's first n allocations fail the same way (a call here replaces it), and
 * the library says so once on stderr. */
tk_status tk_debug_fail_allocations(uint32_t skip, uint32_t count);
/* Test hook: the device memory the library holds now, in bytes, over all devices: the
 * per-device ziggurat state (held until the process ends) and the live alias tables. */
tk_status tk_debug_device_bytes(uint64_t *bytes);
/* Test and benchmark hook: sets a launch tunable for every later call in the process (the
 * defaults, read from TK_* environment variables at first use, are the measured best).
 * Results never depend on them; they choose among launch shapes that compute the same
 * values.  `name` and the accepted values:
 *   "store_nt" 0|1        non-temporal 16-byte stores in the streaming fills (TK_STORE=nt)
 *   "max_blocks" 1..2^31-1  grid cap of the streaming fills, which then stride (TK_MAX_BLOCKS)
 *   "unroll" 1|2|4        16-byte vectors per lane per tile in the streaming fills (TK_UNROLL)
 *   "choice_tiles" 1|2|4|8  4 KiB tiles per choice work-group (TK_CHOICE_TILES)
 *   "exp_tiles" 1|2|4     tiles per exponential work-group (TK_EXP_TILES)
 *   "zig_tiles" 1|2|4|8|16  tiles per ziggurat table-pass work-group (TK_ZIG_TILES)
 *   "zig_lds" 0|1         ziggurat layer gathers from an LDS copy or from L1/L2 (TK_ZIG_TABLE)
 *   "zig_fused" 0|1       ziggurat misses finished in the table pass or a second kernel
 *                         (TK_ZIG_MODE; tk_debug_set_normal_f64_mode overrides it)
 *   "philox_lds" 0|1      Philox fills at word offsets 1..3 by the LDS tile kernel (1) or
 *                         the overlapping-wave kernel (0) (TK_PHILOX=lds|overlap)
 *   "pair_lds" 0|1        lowbias32 Box-Muller fills at odd starts by the pair tile kernel,
 *                         which passes each wave's first value on through LDS (1), or with
 *                         every wave computing the value after it itself (0)
 *                         (TK_PAIRS=lds|wave)
 *   "lds_pad" 0..65536    dynamic LDS bytes allocated per work-group of every fill but the
 *                         ziggurat (for choice, on top of its table), which caps the groups a
 *                         compute unit holds at once (TK_LDS_PAD; unset: each fill's measured
 *                         default, 24 or 32 KiB for the integer fills, else none)
 *   "zig_lds_pad" 0..65536  the same for the ziggurat table pass (TK_ZIG_LDS_PAD)
 *   "const_work" 0..4096  dependent integer steps per lane before each store of
 *                         tk_fill_constant_u32 (TK_CONST_WORK; 0 = none): the spacing of
 *                         the store-ceiling measurement
 * A negative value restores the environment's setting.  Unknown names or values: TK_EINVAL.
 * Not synchronized with launches in flight on other threads beyond each value being read
 * atomically. */
tk_status tk_debug_set_tunable(const char *name, int64_t value);

#ifdef __cplusplus
}
#endif
#endif
