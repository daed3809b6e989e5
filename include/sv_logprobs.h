/*
 * sv_logprobs.h -- C ABI of the operators on given tokens' log-probabilities, for
 * AMD MI355X (gfx950): what a serving reply, the scoring of a rollout and a policy
 * step read from logits [N, V].  Same library (libspec_verify.so).
 *
 *   sv_logprobs       log-probabilities of given tokens, the rows' entropies and
 *                     their largest alternatives
 *   sv_logprobs_grad  the gradient of the logits from those of the log-probabilities
 *                     and entropies
 *
 * Both calls enqueue on `stream` (a hipStream_t; NULL = default stream) and return
 * without synchronising; they allocate nothing and keep no state between calls,
 * so they can be captured in HIP graphs.  Argument errors return a negative
 * SV_ERR_* code (spec_verify.h) before anything is enqueued; data errors set
 * status bits (SV_HEAD_* of sv_head.h).  Results are deterministic: every sum runs
 * in a fixed order.  Device pointers are caller-owned and on the current device.
 * The workspace is scratch memory of at least sv_logprobs_workspace_bytes of the
 * shape, 256-byte aligned, with any contents, before and after; calls that share
 * one must not overlap in time.
 */
#ifndef SV_LOGPROBS_H
#define SV_LOGPROBS_H

#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"
#include "sv_head.h"

#ifdef __cplusplus
extern "C" {
#endif

/* largest number of alternatives of a row */
#define SV_LOGPROBS_MAX_TOP 32

/* ------------------------------------------------- log-probabilities of tokens
 * y[n,v] = logits[n,v] / T, lse_n = ln sum_v exp(y[n,v]), p[n,v] = exp(y[n,v] - lse_n):
 *   logp_n    = y[n, t_n] - lse_n                  (never above 0)
 *   entropy_n = lse_n - sum_v p[n,v] y[n,v]        (never below 0)
 * and the `top` largest logits in the order (value descending, index ascending, -0 equal
 * to +0): top_logp[n,j] = y - lse_n and top_idx[n,j].  Tokens of probability 0 (logits of
 * -inf, as a mask leaves them) have no part in the sums and are no alternatives: where a
 * row has fewer than `top` others, (-inf, -1) follows.
 * norm is the normaliser in two parts, the rows' largest logits and then their ln sum_v exp((logits[n,v] -
 * largest) / T): unlike lse, their sum, it keeps its precision where logits are large, and
 * the gradient reads it.
 * Rows whose token is ignore_index are left out, whatever they hold (their first entries are read
 * all the same, before the token is known): logp = entropy = lse = norm = 0, status 0,
 * alternatives (-inf, -1).  A row with a data error (its token outside the
 * vocabulary, a logit NaN or +inf, or all -inf) has its bits in status, NaN in logp, entropy,
 * lse, norm and top_logp, and -1 in top_idx.  Sums are fp32 over at most 32 terms and fp64
 * beyond.
 */
typedef struct {
    int32_t N;              /* rows, 0 .. SV_HEAD_MAX_N (0: nothing to do) */
    int32_t V;              /* vocabulary, 1 .. SV_HEAD_MAX_V */
    int32_t dtype;          /* logits: SV_F32 or SV_BF16 */
    int32_t top;            /* alternatives, 0 .. SV_LOGPROBS_MAX_TOP */
    int64_t row_stride;     /* elements between rows of logits; 0 means V */
    float temperature;      /* T > 0, and log2(e) / T finite */
    int32_t ignore_index;
} sv_logprobs_shape_t;

/* 0 where a shape needs none (the workspace may then be NULL), or is refused */
size_t sv_logprobs_workspace_bytes(const sv_logprobs_shape_t *shape);

/* logits [N, V]; tokens [N] int32; logp [N], entropy [N], lse [N] and norm [2, N] fp32 and
 * status [N] int32, each but logp may be NULL; top_logp [N, top] fp32 and top_idx [N, top]
 * int32, required where top > 0.  N = 0: returns SV_OK, enqueues nothing and leaves every
 * output untouched. */
int sv_logprobs(const sv_logprobs_shape_t *shape, const void *logits, const int32_t *tokens, float *logp,
                float *entropy, float *lse, float *norm, int32_t *status, float *top_logp, int32_t *top_idx,
                void *workspace, size_t workspace_bytes, void *stream);

/* --------------------------------------------------------------- their gradient
 * From g_n, the gradient of logp_n, and h_n, that of entropy_n (0 without one):
 *   grad[n,v] = (1/T) (g_n ([v = t_n] - p[n,v]) - h_n p[n,v] (ln p[n,v] + entropy_n))
 * with p from norm, all of the same logits, tokens and temperature as in sv_logprobs.  Rows
 * that are left out, rows whose token is outside the vocabulary and rows whose norm is not
 * finite (those with a data error) have a gradient of 0 whatever their g and h, and are not
 * read.  Of other rows a g or h that is not finite makes every entry NaN or infinite; entries
 * beyond the gradient's type are infinite (magnitudes of g and h up to 1e36, at any temperature).
 */
typedef struct {
    int32_t N, V;           /* as above */
    int32_t dtype;          /* logits: SV_F32 or SV_BF16 */
    int32_t grad_dtype;     /* gradient: SV_F32 or SV_BF16 */
    int64_t row_stride;     /* elements between rows of logits; 0 means V */
    int64_t grad_stride;    /* elements between rows of the gradient; 0 means V */
    float temperature;
    int32_t ignore_index;
} sv_logprobs_grad_shape_t;

/* norm [2, N], grad_logp [N] fp32; grad_entropy [N] fp32 or NULL; entropy [N] fp32, required
 * with grad_entropy; grad [N, V], all of it written (nothing between V and a stride).  grad
 * may be the logits' own memory where type and stride are theirs; it may not overlap them
 * otherwise. */
int sv_logprobs_grad(const sv_logprobs_grad_shape_t *shape, const void *logits, const int32_t *tokens,
                     const float *norm, const float *entropy, const float *grad_logp, const float *grad_entropy,
                     void *grad, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SV_LOGPROBS_H */
