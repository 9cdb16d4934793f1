/*
 * gemm_ffn.h -- the operators of a feed-forward block around and within its
 * products, as part of libgemm_gb300.so:
 *
 *   RMS norm      t = x + residual;  y = t / sqrt(mean t^2 + eps) * gamma, in the
 *                 rows' type or in 8 bits with scales, and its gradients
 *   8 bits        a matrix as e4m3 numbers with a scale for each 128 elements of a
 *                 row, or for each 128 x 128 elements; as it stands or transposed
 *
 * Types, ownership, threading and errors as in gemm.h and gemm_train.h: matrices
 * are row-major; calls are asynchronous on the caller's stream, allocate nothing,
 * can be captured into a CUDA graph, and report argument problems before any device
 * work is queued:
 *   GEMM_ERR_INVALID_ARG  a size out of range, a row stride below the row's length,
 *                         a NULL pointer where one is needed, another device current
 *   GEMM_ERR_UNSUPPORTED  an unknown type, activation or kind of scales
 *   GEMM_ERR_ALIGNMENT    a pointer (or a size of a product's operand) that is not
 *                         aligned as the call needs it
 * A plan is used with the device current on which it was made, by one thread at a
 * time.  All sums and statistics are fp32; a result is rounded once, to nearest even.
 * Results do not depend on the schedule: the same inputs give the same bits.
 */
#ifndef GB300_GEMM_FFN_H
#define GB300_GEMM_FFN_H

#include "gemm.h"
#include "gemm_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * 8-bit matrices.  An e4m3 number has 4 exponent and 3 mantissa bits, its largest
 * value is 448.  128 consecutive elements of a row share an fp32 scale (the last
 * group of a row may be shorter), or 128 x 128 elements do:
 *     GEMM_SCALE_ROW     scales[i][g]      of elements i, 128 g .. 128 g + 127
 *     GEMM_SCALE_SQUARE  scales[i/128][g]  of elements i, 128 g .. 128 g + 127
 * Scales are row-major fp32, ceil(cols / 128) a row.  The number an element stands
 * for is its e4m3 value times its scale.  Conversion, in fp32:
 *     scale = max(largest |value| * fl(1/448), 2^-126)
 *     q     = value * fl(1 / scale), rounded to nearest even, at most 448 in size
 * NaN takes no part in the largest value and stays NaN in its place; a group with an
 * infinity gets the scale infinity, its other elements 0.
 */
typedef enum {
    GEMM_SCALE_ROW = 0,
    GEMM_SCALE_SQUARE = 1
} gemm_scale_t;

/* ------------------------------------------------------------------ RMS norm */

typedef struct gemm_rms_plan *gemm_rms_plan_t;

/*
 * A plan for up to max_rows rows of `cols` elements (1 <= cols <= 2^30,
 * 0 <= max_rows < 2^31).  elem: type of the rows; weight_elem: type of gamma and its
 * gradient, either elem or GEMM_ELEM_F32 (else GEMM_ERR_UNSUPPORTED).  The plan owns
 * the workspace of the weight's gradient: one stream at a time.
 */
gemm_status_t gemm_rms_plan_create(int64_t max_rows, int64_t cols, gemm_elem_t elem,
                                   gemm_elem_t weight_elem, gemm_rms_plan_t *plan);

/*
 * For each of `rows` rows: t = x + residual, rounded to the rows' type (residual NULL:
 * t = x), rstd = 1 / sqrt(mean t^2 + eps), y = t * rstd * gamma (gamma NULL = ones).
 * total (NULL: not kept) receives t, rstd (NULL: not kept) one fp32 value a row: what
 * the backward call takes.  eps >= 0.  total and y may each be x or residual (same
 * stride), but not the same matrix; matrices overlap in no other way.
 */
gemm_status_t gemm_rms_forward(gemm_rms_plan_t plan, int64_t rows, const void *x, int64_t ldx,
                               const void *residual, int64_t ldr, const void *gamma, float eps,
                               void *total, int64_t ldt, void *y, int64_t ldy, float *rstd,
                               void *stream);

/*
 * As gemm_rms_forward, with y (unrounded) converted to 8 bits: q (rows x cols bytes,
 * starts ldq apart) and its scales by rows (starts lds >= ceil(cols / 128) apart).
 */
gemm_status_t gemm_rms_forward_fp8(gemm_rms_plan_t plan, int64_t rows, const void *x, int64_t ldx,
                                   const void *residual, int64_t ldr, const void *gamma, float eps,
                                   void *total, int64_t ldt, void *q, int64_t ldq, float *scales,
                                   int64_t lds, float *rstd, void *stream);

/*
 * With th = total * rstd and g = dy * gamma:
 *     dx     = rstd * (g - th * sum(g * th) / cols) + dtotal     (dtotal NULL = zeros)
 *     dgamma = sum over rows of dy * th
 * dx is the gradient of x and of residual; dtotal is the gradient that reaches the sum
 * on its other way.  gamma NULL = ones.  dx and dgamma may each be NULL (not
 * computed); they are overwritten, and rows == 0 gives zero dgamma.  dx may be dy,
 * dtotal or total (same stride); matrices overlap in no other way.
 */
gemm_status_t gemm_rms_backward(gemm_rms_plan_t plan, int64_t rows, const void *total, int64_t ldt,
                                const void *gamma, const float *rstd, const void *dy, int64_t lddy,
                                const void *dtotal, int64_t lddt, void *dx, int64_t lddx,
                                void *dgamma, void *stream);

/* Free a plan and its device memory.  NULL is a no-op. */
gemm_status_t gemm_rms_plan_destroy(gemm_rms_plan_t plan);

/* ------------------------------------------------------------------ conversion to 8 bits */

/*
 * x (rows x cols of `elem`) to 8 bits: q and scales of x, or of its transpose where
 * `transpose` is 1 (q is then cols x rows).  ldq, lds: row strides of q (in bytes) and
 * of the scales.  rows, cols: 0 to 2^31 - 1, at most 2^30 squares of 128 x 128.  No plan is
 * needed; the call goes to the current device.
 */
gemm_status_t gemm_fp8_quantize(int64_t rows, int64_t cols, gemm_elem_t elem, const void *x,
                                int64_t ldx, gemm_scale_t kind, int32_t transpose, void *q,
                                int64_t ldq, float *scales, int64_t lds, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GB300_GEMM_FFN_H */
