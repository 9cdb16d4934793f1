/*
 * gemm_train.h -- the operators around the products of a training step, as part
 * of libgemm_gb300.so:
 *
 *   embedding     out[t] = scale * table[ids[t]], and the gradient of the table
 *   layer norm    y = (x - mean) / sqrt(var + eps) * gamma + beta, and the
 *                 gradients of x, gamma and beta
 *   distillation  tau^2 * KL(teacher's top entries || softmax(logits / tau)) per
 *                 row, and its gradient in the logits
 *
 * They take and leave matrices as the products of gemm.h do: row-major, rows of
 * `cols` contiguous elements whose starts are `ld` elements apart (ld >= cols),
 * so the logits of a product whose N was padded to a multiple of 8 are used in
 * place.  Elements between cols and ld are never written, and take no part in a
 * result; the norm may read those within 16 bytes of a row that is not the matrix'
 * first or last.
 *
 * Types: fp16, bf16 or fp32 elements (gemm_elem_t).  All sums, softmax and norm
 * statistics are fp32; a result is rounded once (to nearest even) to its type.
 *
 * Ownership, threading, errors: as in gemm.h.  A plan is created on the current
 * device for a largest size, owns its device memory (workspace and error word),
 * and must be used with that device current and on one stream at a time.  The
 * calls are asynchronous on the caller's stream, allocate nothing, and can be
 * captured into a CUDA graph.  Argument problems are reported before any device
 * work is queued:
 *   GEMM_ERR_INVALID_ARG  a size out of the plan's range, ld < cols, a NULL
 *                         pointer where one is needed, another device current
 *   GEMM_ERR_UNSUPPORTED  an unknown type
 *   GEMM_ERR_ALIGNMENT    a pointer that is not aligned to its element's size
 * Any stride is taken; rows whose starts are 16-byte aligned are fastest.
 * An index out of its range cannot be seen before the kernel reads it: the
 * kernel skips it, sets the plan's error word, and the plan's check call reports
 * GEMM_ERR_INDEX.
 *
 * Results do not depend on the schedule: the same inputs give the same bits.
 */
#ifndef GB300_GEMM_TRAIN_H
#define GB300_GEMM_TRAIN_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GEMM_ELEM_F16 = 0,
    GEMM_ELEM_BF16 = 1,
    GEMM_ELEM_F32 = 2
} gemm_elem_t;

typedef enum {
    GEMM_INDEX_I32 = 0,
    GEMM_INDEX_I64 = 1
} gemm_index_t;

/* ------------------------------------------------------------------ layer norm */

typedef struct gemm_norm_plan *gemm_norm_plan_t;

/*
 * A plan for up to max_rows rows of `cols` elements (1 <= cols <= 2^30,
 * 0 <= max_rows < 2^31).  elem: type of x, y, dy and dx; weight_elem: type of
 * gamma, beta and their gradients, either elem or GEMM_ELEM_F32 (else
 * GEMM_ERR_UNSUPPORTED).
 */
gemm_status_t gemm_norm_plan_create(int64_t max_rows, int64_t cols, gemm_elem_t elem,
                                    gemm_elem_t weight_elem, gemm_norm_plan_t *plan);

/*
 * For each of `rows` rows: mean = sum x / cols, var = sum (x - mean)^2 / cols,
 * rstd = 1 / sqrt(var + eps), y = (x - mean) * rstd * gamma + beta.
 * gamma NULL = ones, beta NULL = zeros; mean, rstd: `rows` fp32 values each,
 * which the backward call takes, or NULL.  eps >= 0.  y may be x (same stride).
 */
gemm_status_t gemm_norm_forward(gemm_norm_plan_t plan, int64_t rows, const void *x, int64_t ldx,
                                const void *gamma, const void *beta, float eps, void *y,
                                int64_t ldy, float *mean, float *rstd, void *stream);

/*
 * With xh = (x - mean) * rstd and g = dy * gamma:
 *     dx     = rstd * (g - sum g / cols - xh * sum(g * xh) / cols)
 *     dgamma = sum over rows of dy * xh        dbeta = sum over rows of dy
 * gamma NULL = ones.  dx, dgamma and dbeta may each be NULL (not computed); they
 * are overwritten, and rows == 0 gives zero dgamma and dbeta.  dx may be dy or x
 * (same stride).
 */
gemm_status_t gemm_norm_backward(gemm_norm_plan_t plan, int64_t rows, const void *x, int64_t ldx,
                                 const void *gamma, const float *mean, const float *rstd,
                                 const void *dy, int64_t lddy, void *dx, int64_t lddx,
                                 void *dgamma, void *dbeta, void *stream);

/*
 * Set the limit, in nanoseconds, after which a wait in a kernel of this plan
 * gives up (default 2e9, 2e4 to 4e9).  ns == 0 restores the default.  The calls
 * that follow (graphs captured from then on) have it.
 */
gemm_status_t gemm_norm_plan_set_timeout(gemm_norm_plan_t plan, uint64_t ns);

/*
 * Test hook for failure reporting: in every `every`-th block (1 = all) the copies
 * of rows wait for `extra_bytes` (a multiple of 16, at most 4096) more than they
 * bring, so their waits run out, the kernel returns, and the check below reports
 * GEMM_ERR_DEVICE_TIMEOUT; the results are undefined.  The GPU context stays
 * usable.  0 restores normal operation.  Few, short and very wide rows, which are
 * not copied but loaded, have no such waits.
 */
gemm_status_t gemm_norm_plan_set_wait_test(gemm_norm_plan_t plan, uint32_t extra_bytes,
                                           uint32_t every);

/*
 * Synchronise `stream`, then read and clear the plan's error word:
 * GEMM_ERR_DEVICE_TIMEOUT if a kernel of this plan gave up on a wait, GEMM_ERR_CUDA
 * if the stream reported an error, else GEMM_OK.
 */
gemm_status_t gemm_norm_plan_check(gemm_norm_plan_t plan, void *stream);

/* Free a plan and its device memory.  NULL is a no-op. */
gemm_status_t gemm_norm_plan_destroy(gemm_norm_plan_t plan);

/* ------------------------------------------------------------------ embedding */

typedef struct gemm_embed_plan *gemm_embed_plan_t;

/*
 * A plan for a table of `vocab` rows of `dim` elements and up to max_tokens
 * tokens a call (1 <= vocab < 2^31, 1 <= dim <= 2^30, 0 <= max_tokens < 2^31).
 * elem: type of the table, of out and of dout; grad_elem: type of the table's
 * gradient, either elem or GEMM_ELEM_F32 (else GEMM_ERR_UNSUPPORTED).
 */
gemm_status_t gemm_embed_plan_create(int64_t vocab, int64_t dim, int64_t max_tokens,
                                     gemm_elem_t elem, gemm_elem_t grad_elem,
                                     gemm_embed_plan_t *plan);

/*
 * out[t] = scale * table[ids[t]] for `tokens` contiguous ids.  A token equal to
 * `padding` gives a row of zeros (padding < 0 may be used as an id for that
 * purpose too; padding outside [0, vocab) and never used = no padding).  Any
 * other id outside [0, vocab) is reported by gemm_embed_plan_check, and its row
 * is zeros.
 */
gemm_status_t gemm_embed_forward(gemm_embed_plan_t plan, int64_t tokens, const void *ids,
                                 gemm_index_t id_type, int64_t padding, const void *table,
                                 int64_t ldt, float scale, void *out, int64_t ldo, void *stream);

/*
 * dtable[v] = scale * sum of dout[t] over the tokens t with ids[t] == v, summed in
 * fp32 in an order that depends on the ids alone; padding and out-of-range tokens
 * take no part.  accumulate == 0: every row of dtable is written (rows without a
 * token as zeros); accumulate == 1: the sums are added to dtable (in fp32, then
 * rounded once), and rows without a token are not touched.  In fp32 that addition
 * takes numbers below the smallest normal one as zeros.
 */
gemm_status_t gemm_embed_backward(gemm_embed_plan_t plan, int64_t tokens, const void *ids,
                                  gemm_index_t id_type, int64_t padding, const void *dout,
                                  int64_t ldo, float scale, void *dtable, int64_t ldt,
                                  int32_t accumulate, void *stream);

/*
 * Synchronise `stream`, then read and clear the plan's error word: GEMM_ERR_INDEX
 * if a call since the last check met an id outside its range, GEMM_ERR_CUDA if
 * the stream reported an error, else GEMM_OK.
 */
gemm_status_t gemm_embed_plan_check(gemm_embed_plan_t plan, void *stream);

/* Free a plan and its device memory.  NULL is a no-op. */
gemm_status_t gemm_embed_plan_destroy(gemm_embed_plan_t plan);

/* ------------------------------------------------------------------ distillation */

typedef struct gemm_distill_plan *gemm_distill_plan_t;

/*
 * What the teacher left of its distribution: for each row its `top` entries, a
 * token id and a logit each.  A negative id is no entry (rows with fewer entries
 * than top), in any place.  The ids of a row are usually distinct; equal ones add
 * their probabilities.
 *
 * With tau the temperature, the teacher's probabilities are
 *     p_j = exp(values_j / tau - L)
 * where L = lse[row] if lse is given (log of the sum of exp(logit / tau) over the
 * teacher's whole vocabulary: the p_j then sum to less than one), else
 * L = log sum_j exp(values_j / tau) over the row's entries (they sum to one).
 */
typedef struct {
    const void *ids;          /* rows x top, starts ld_ids elements apart */
    const void *values;       /* rows x top, starts ld_values elements apart */
    const float *lse;         /* rows values, or NULL */
    int64_t top;              /* 0 <= top <= the plan's max_top */
    int64_t ld_ids;
    int64_t ld_values;
    gemm_index_t id_type;
    gemm_elem_t value_elem;
} gemm_teacher_t;

/*
 * A plan for up to max_rows rows of logits over `vocab` tokens and up to max_top
 * teacher entries a row (1 <= vocab <= 2^30, 0 <= max_rows < 2^31,
 * 0 <= max_top <= 1024).  elem: type of the logits and of their gradient.
 */
gemm_status_t gemm_distill_plan_create(int64_t max_rows, int64_t vocab, int64_t max_top,
                                       gemm_elem_t elem, gemm_distill_plan_t *plan);

/*
 * For each row, with q = softmax(logits / tau) over the vocabulary:
 *     lse  = log sum_i exp(logits_i / tau)
 *     loss = tau^2 * sum_j p_j * (log p_j - log q_{ids_j})     (0 where p_j = 0)
 * A row is left out where the teacher has no mass (no entry, or -infinity values
 * only) or where no logit is above -infinity: loss 0, lse -infinity, gradient 0.
 * Logits of -infinity (masked tokens) have q = 0, and a logit below -1e30 * tau
 * counts as one (masks of a type's lowest value); NaN logits give NaN.
 * temperature: a normal positive number.  An id >= vocab is reported by gemm_distill_plan_check and
 * taken as no entry.
 */
gemm_status_t gemm_distill_forward(gemm_distill_plan_t plan, int64_t rows, const void *logits,
                                   int64_t ldl, const gemm_teacher_t *teacher, float temperature,
                                   float *loss, float *lse, void *stream);

/*
 * dlogits_i = dloss * tau * (P * q_i - sum of p_j over j with ids_j == i),
 * P = sum_j p_j, from the forward call's lse.  That is a number in fp32: each q_i is
 * as far off, relatively, as lse is absolutely (2^-24 of its size; from 2^22 on no q_i
 * is above one).  dloss: the upstream gradient of each row's loss (`rows` fp32
 * values), or NULL for ones.  dlogits may be logits (same stride).
 */
gemm_status_t gemm_distill_backward(gemm_distill_plan_t plan, int64_t rows, const void *logits,
                                    int64_t ldl, const gemm_teacher_t *teacher, float temperature,
                                    const float *lse, const float *dloss, void *dlogits,
                                    int64_t ldd, void *stream);

/*
 * Both in one call, for a training step whose upstream gradient is known before
 * the loss: each row's logits are read from memory once where they fit on the
 * chip, and the gradient does not go through the rounded lse.
 */
gemm_status_t gemm_distill_forward_backward(gemm_distill_plan_t plan, int64_t rows,
                                            const void *logits, int64_t ldl,
                                            const gemm_teacher_t *teacher, float temperature,
                                            const float *dloss, float *loss, float *lse,
                                            void *dlogits, int64_t ldd, void *stream);

/*
 * Set the limit, in nanoseconds, after which a wait in a kernel of this plan
 * gives up (default 2e9, 2e4 to 4e9).  ns == 0 restores the default.  The calls
 * that follow (graphs captured from then on) have it.
 */
gemm_status_t gemm_distill_plan_set_timeout(gemm_distill_plan_t plan, uint64_t ns);

/*
 * Test hook for failure reporting: in every `every`-th block (1 = all) the copies
 * of logits wait for `extra_bytes` (a multiple of 16, at most 4096) more than they
 * bring, so their waits run out, the kernel returns, and the check below reports
 * GEMM_ERR_DEVICE_TIMEOUT; the results are undefined.  The GPU context stays
 * usable.  0 restores normal operation.  Rows of up to 16 packs of 16 bytes a
 * lane of a warp, and rows that no eight blocks can hold, have no such waits.
 */
gemm_status_t gemm_distill_plan_set_wait_test(gemm_distill_plan_t plan, uint32_t extra_bytes,
                                              uint32_t every);

/*
 * As gemm_embed_plan_check, for the teacher's ids; GEMM_ERR_DEVICE_TIMEOUT if a
 * kernel of this plan gave up on a wait.
 */
gemm_status_t gemm_distill_plan_check(gemm_distill_plan_t plan, void *stream);

/* Free a plan and its device memory.  NULL is a no-op. */
gemm_status_t gemm_distill_plan_destroy(gemm_distill_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* GB300_GEMM_TRAIN_H */
