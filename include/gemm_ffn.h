/*
 * gemm_ffn.h -- the operators of a feed-forward block around and within its
 * products, as part of libgemm_gb300.so:
 *
 *   RMS norm      t = x + residual;  y = t / sqrt(mean t^2 + eps) * gamma, in the
 *                 rows' type or in 8 bits with scales, and its gradients
 *   8 bits        a matrix as e4m3 numbers with a scale for each 128 elements of a
 *                 row, or for each 128 x 128 elements; as it stands or transposed
 *   8-bit product C = A * B^T of such matrices
 *   gated product H = act(X * Wg^T) * (X * Wu^T), and its gradients
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
 * A plan is used with the device current on which it was made, by one thread and on
 * one stream at a time (graphs captured from one plan are replayed one after another).
 * All sums and statistics are fp32; a result is rounded once, to nearest even.
 * Results do not depend on the schedule, nor on where they go: the same inputs give the same
 * bits (inputs that lie elsewhere to the 16-byte boundaries may be summed in another order).
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
 * the backward call takes.  eps >= 0.  The sum of squares is fp32: it has to stay within
 * that type (elements of up to about 1e18; a row beyond has rstd 0), and with eps == 0 a
 * row's mean square may not underflow.  total and y may each be x or residual (same
 * stride), but not the same matrix; matrices overlap in no other way.  Rows are read in
 * 16 aligned bytes, of which at least one is the row's; only a row's own elements are used
 * and written.
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
 * of the scales.  rows, cols: 0 to 2^31 - 1, at most 2^29 squares of 128 x 128.  No plan is
 * needed; the call goes to the current device.
 */
gemm_status_t gemm_fp8_quantize(int64_t rows, int64_t cols, gemm_elem_t elem, const void *x,
                                int64_t ldx, gemm_scale_t kind, int32_t transpose, void *q,
                                int64_t ldq, float *scales, int64_t lds, void *stream);

/* ------------------------------------------------------------------ 8-bit product */

typedef struct gemm_fp8_plan *gemm_fp8_plan_t;

/*
 * A plan for C[i][j] = sum over groups g of a_scales[i][g] * sb(j, g) * sum over k in g of
 * A[i][k] * B[j][k], with A M x K and B N x K (e4m3, K-contiguous) and C M x N of `out`
 * (GEMM_ELEM_F16 or GEMM_ELEM_BF16).  A's scales go by rows, B's by b_scales: squares
 * (weights) or rows (where both are activations).  K has to be a multiple of 16 and N of
 * 8 (GEMM_ERR_ALIGNMENT); M, N <= 2^31 - 257, K <= 2^31 - 129, and at most 2^27 tiles of
 * 128 x 128 of C.  Any other K (a weight gradient's tokens): rows of the next multiple of 16
 * bytes, zeros behind the K elements in both operands, to whose front gemm_fp8_quantize
 * converts (ldq); the scales of K elements are as many.
 * The scales of a group are multiplied in fp32 with each other (squares), or one after the other
 * with the group's sum (rows): what leaves that type's range on the way is lost.
 */
gemm_status_t gemm_fp8_plan_create(int64_t M, int64_t N, int64_t K, gemm_elem_t out,
                                   gemm_scale_t b_scales, gemm_fp8_plan_t *plan);

/*
 * Queue the product.  A, B and C contiguous and 16-byte aligned; scales contiguous
 * (M x ceil(K/128), and N or ceil(N/128) x ceil(K/128)), 4-byte aligned.  K == 0 writes
 * zeros.  C overlaps no operand.
 */
gemm_status_t gemm_fp8_run(gemm_fp8_plan_t plan, const void *A, const float *a_scales, const void *B,
                           const float *b_scales, void *C, void *stream);

/*
 * As gemm_plan_set_timeout, gemm_plan_set_wait_test, gemm_plan_check and
 * gemm_plan_destroy of gemm.h.
 */
gemm_status_t gemm_fp8_plan_set_timeout(gemm_fp8_plan_t plan, uint64_t ns);
gemm_status_t gemm_fp8_plan_set_wait_test(gemm_fp8_plan_t plan, uint32_t extra_bytes);
gemm_status_t gemm_fp8_plan_check(gemm_fp8_plan_t plan, void *stream);
gemm_status_t gemm_fp8_plan_destroy(gemm_fp8_plan_t plan);

/* ------------------------------------------------------------------ gated product */

typedef struct gemm_gated_plan *gemm_gated_plan_t;

/*
 * A plan for H = act(X * Wg^T) * (X * Wu^T): X is M x K, W = [Wg; Wu] is 2F x K (rows
 * 0 .. F-1 the gate's weights, F .. 2F-1 the other's) and H is M x F, all of `elem`
 * (GEMM_ELEM_F16 or GEMM_ELEM_BF16) and contiguous.  F and K have to be multiples of 8
 * (GEMM_ERR_ALIGNMENT); M, K < 2^31, F < 2^30, and at most 2^27 tiles of 128 x 64 of H.
 * act: GEMM_ACT_NONE, _RELU, _GELU or _SILU.
 */
gemm_status_t gemm_gated_plan_create(int64_t M, int64_t F, int64_t K, gemm_elem_t elem,
                                     gemm_activation_t act, gemm_gated_plan_t *plan);

/*
 * Queue H.  gate_up (M x 2F) receives both products side by side, rounded to the type:
 * what the backward call takes; NULL: not kept.  H itself is of the unrounded products.
 * K == 0 gives zeros.  Pointers 16-byte aligned; outputs overlap no operand.
 */
gemm_status_t gemm_gated_forward(gemm_gated_plan_t plan, const void *X, const void *W, void *H,
                                 void *gate_up, void *stream);

/*
 * Gradients, with g and u the halves of gate_up's rows:
 *     dgate_up = [dH * u * act'(g), dH * act(g)]      (M x 2F, rounded to the type)
 *     dX = dgate_up * W                               (M x K)
 *     dW = dgate_up^T * X                             (2F x K)
 * dX and dW may each be NULL (not computed; W and X are then not read).  dgate_up may
 * be gate_up; outputs overlap no other operand.  dX and dW are products of gemm.h over
 * dgate_up.  act'(0) of ReLU is 0.
 */
gemm_status_t gemm_gated_backward(gemm_gated_plan_t plan, const void *X, const void *W,
                                  const void *gate_up, const void *dH, void *dgate_up, void *dX,
                                  void *dW, void *stream);

/* As for gemm_fp8_plan_t (the backward products' waits included). */
gemm_status_t gemm_gated_plan_set_timeout(gemm_gated_plan_t plan, uint64_t ns);
gemm_status_t gemm_gated_plan_set_wait_test(gemm_gated_plan_t plan, uint32_t extra_bytes);
gemm_status_t gemm_gated_plan_check(gemm_gated_plan_t plan, void *stream);
gemm_status_t gemm_gated_plan_destroy(gemm_gated_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* GB300_GEMM_FFN_H */
