/*
 * sv_head.h -- C ABI of the vocabulary-head operators, for AMD MI355X (gfx950):
 * the steps before spec_verify.h and around sv_kd.h that start from hidden rows
 * [N, H] and the head's weight [V, H] instead of logits [N, V].  Same library
 * (libspec_verify.so).
 *
 *   sv_act8_pack / sv_act8_unpack  hidden rows in 8 bits with a scale per row
 *   sv_head_logits                 logits of hidden rows under a head held in
 *                                  8-bit integers, as spec_verify takes them
 *   sv_head_ce                     softmax cross entropy of hidden rows under the
 *                                  head, with the gradients of both
 *   sv_head_kd                     sv_kd's distillation loss the same way
 *
 * The online fine-tuning of the drafter (Notion post "Power Up Speculative
 * Decoding in RL": the MTP drafter is trained with SFT beside the policy) and
 * the distillation over the stored top-32 (ReSpec notes, "4 . G2" and "5 . G3")
 * both end in a product with a vocabulary head; the losses here form its logits
 * in pieces of the vocabulary and keep none of them.
 *
 * All calls enqueue on `stream` (a hipStream_t; NULL = default stream) and return
 * without synchronising; they allocate nothing and keep no state between calls,
 * so they can be captured in HIP graphs.  Argument errors return a negative
 * SV_ERR_* code (spec_verify.h) before anything is enqueued; data errors set
 * status bits.  Results are deterministic: every sum runs in a fixed order.
 * Device pointers are caller-owned and on the current device.  A workspace is
 * scratch memory of at least the *_workspace_bytes of the shape, 256-byte
 * aligned, with any contents, before and after; calls that share one must not
 * overlap in time.
 */
#ifndef SV_HEAD_H
#define SV_HEAD_H

#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element type of rows held as 8-bit codes with a scale per row (beside
 * SV_F32 and SV_BF16 of sv_dtype_t) */
#define SV_I8 2

/* largest hidden width: the int32 sum of H products of two codes of magnitude
 * 127 stays below 2^31 */
#define SV_HEAD_MAX_H 131072
/* largest number of rows and largest vocabulary of the losses */
#define SV_HEAD_MAX_N 1048576
#define SV_HEAD_MAX_V 16777216

/* ---------------------------------------------------------------- 8-bit rows
 *   scale[n] = fl(max_k |x[n,k]| / 127)
 *   codes[n,k] = clamp(round_to_even(x[n,k] / scale[n]), -127, 127), exactly
 *                rounded also where scale[n] is subnormal; 0 where it is 0
 *   unpacked y[n,k] = codes[n,k] * scale[n]
 * A row holding a NaN or an infinity gets scale NaN and codes 0 (unpacked: NaN).
 * x [N, H] (SV_F32 or SV_BF16) with row stride x_stride elements, codes [N, H]
 * int8 with row stride codes_stride bytes, scale [N] fp32, y [N, H] contiguous in
 * y_dtype; a stride of 0 means H.  Elements between H and a stride are not written.
 * N = 0: returns SV_OK and enqueues nothing.
 */
int sv_act8_pack(int32_t N, int32_t H, int32_t dtype, const void *x, int64_t x_stride, int8_t *codes,
                 int64_t codes_stride, float *scale, void *stream);
int sv_act8_unpack(int32_t N, int32_t H, const int8_t *codes, int64_t codes_stride, const float *scale,
                   int32_t y_dtype, void *y, void *stream);

/* ------------------------------------------------------------ 8-bit head logits
 *   logits[n,v] = scale_x[n] * scale_w[v] * sum_k cx[n,k] cw[v,k]
 * The sum is exact (int32).  It, the product of the two scales and the product of
 * both are each rounded to fp32 once, the last to bf16 as well where the logits are bf16.  cx is either given (hidden_dtype SV_I8,
 * with hidden_scale) or formed from fp32 or bf16 rows as sv_act8_pack does.
 */
typedef struct {
    int32_t N;              /* hidden rows, >= 0 (0: nothing to do) */
    int32_t H;              /* hidden width, 1 .. SV_HEAD_MAX_H */
    int32_t V;              /* vocabulary entries, 1 .. SV_HEAD_MAX_V */
    int32_t hidden_dtype;   /* SV_F32, SV_BF16 or SV_I8 */
    int32_t out_dtype;      /* SV_F32 or SV_BF16 */
    int64_t hidden_stride;  /* elements between hidden rows; 0 means H */
    int64_t weight_stride;  /* bytes between weight code rows; 0 means H */
    int64_t out_stride;     /* elements between logits rows; 0 means V */
} sv_logits_shape_t;

size_t sv_head_logits_workspace_bytes(const sv_logits_shape_t *shape);

/* hidden [N, H]; hidden_scale [N] fp32 (SV_I8 only, else ignored); weight_codes
 * [V, H] int8; weight_scale [V] fp32; logits [N, V] (out_dtype).  A row whose
 * scale is NaN gives NaN logits, which spec_verify reports. */
int sv_head_logits(const sv_logits_shape_t *shape, const void *hidden, const float *hidden_scale,
                   const int8_t *weight_codes, const float *weight_scale, void *logits, void *workspace,
                   size_t workspace_bytes, void *stream);

/* ----------------------------------------------------------------- losses
 * z[n,v] = (1/T) sum_k x[n,k] w[v,k], lse_n = ln sum_v exp(z[n,v]).
 *
 * sv_head_ce:  nll_n = lse_n - z[n, t_n],  loss = sum_n u_n nll_n,
 *              dz[n,v] = u_n (exp(z[n,v] - lse_n) - [v = t_n])
 *   with u_n = row_weight[n] (1 without one; any finite value, so an advantage
 *   makes it a policy-gradient step).  Rows whose target is ignore_index are left
 *   out: nll = lse = 0, status 0, no gradient.
 * sv_head_kd:  sv_kd's formulas with z for its drafter logits (T = 1): KL_n over
 *   the stored 32, u_n = the clipped group-normalised reward.
 * Gradients of both: dx[n,k] = (1/T) sum_v dz[n,v] w[v,k],
 *                    dw[v,k] = (1/T) sum_n dz[n,v] x[n,k].
 * Products of bf16 operands are summed in fp32; for them dz is rounded to bf16, as
 * it is an operand of the gradients' products (their error: 0.0020 to 0.0028 of the
 * norm, where the rounding of the results alone is 0.0015 to 0.0017).  Up to 32
 * rows, and with SV_GRAD_TWO_TERMS at any number, it is the sum of two bf16 numbers
 * (0.0015 to 0.0017; a second product of each gradient beyond 32 rows).  Everything
 * else is fp32 or fp64.
 */
#define SV_GRAD_HIDDEN 1
#define SV_GRAD_WEIGHT 2
#define SV_GRAD_TWO_TERMS 4   /* with one of the others; changes nothing for fp32 */

/* status bits of sv_head_ce, per row (sv_head_kd: the SV_KD_* bits of sv_kd.h) */
#define SV_HEAD_BAD_TARGET 1   /* the target is neither ignore_index nor in [0, V) */
#define SV_HEAD_NAN 2          /* a logit of the row is NaN */
#define SV_HEAD_POSINF 4       /* a logit of the row is +inf */
#define SV_HEAD_EMPTY 8        /* every logit of the row is -inf */
#define SV_HEAD_BAD_WEIGHT 16  /* row_weight is NaN or infinite */

typedef struct {
    int32_t N;              /* rows, 0 .. SV_HEAD_MAX_N (0: nothing to do) */
    int32_t H;              /* hidden width, 1 .. SV_HEAD_MAX_H */
    int32_t V;              /* vocabulary, 1 .. SV_HEAD_MAX_V */
    int32_t dtype;          /* SV_F32 or SV_BF16: the weight and both gradients */
    int32_t hidden_dtype;   /* dtype, or SV_I8: codes with hidden_scale (the rows' values
                               are codes * scale, in the gradient of the weight too) */
    int32_t grads;          /* SV_GRAD_* bits of the gradients to compute */
    int64_t hidden_stride;  /* elements between hidden rows; 0 means H */
    int64_t weight_stride;  /* elements between weight rows; 0 means H */
    float temperature;      /* T > 0 (sv_head_kd: must be 1) */
    int32_t ignore_index;   /* sv_head_ce */
    int32_t S;              /* sv_head_kd: samples, >= 1 when N > 0 */
    int32_t group;          /* sv_head_kd: samples per reward group, >= 1, dividing S */
    float w_max;            /* sv_head_kd: clip of the weight, > 0 (+inf: no clip) */
} sv_head_shape_t;

size_t sv_head_ce_workspace_bytes(const sv_head_shape_t *shape);
size_t sv_head_kd_workspace_bytes(const sv_head_shape_t *shape);

/* hidden [N, H]; hidden_scale [N] fp32 (SV_I8 only, else ignored); weight [V, H];
 * targets [N] int32; row_weight [N] fp32 or NULL.
 * nll, lse [N] fp32 (lse may be NULL) and status [N] int32 (may be NULL): NaN, NaN
 * and the bits for a row with a data error, which adds nothing to the loss and
 * the gradients; loss [1] fp32, summed in fp64; grad_hidden [N, H] and grad_weight
 * [V, H], contiguous, in dtype, required where shape->grads asks for them.
 * N = 0: returns SV_OK, enqueues nothing and leaves every output untouched. */
int sv_head_ce(const sv_head_shape_t *shape, const void *hidden, const float *hidden_scale, const void *weight,
               const int32_t *targets, const float *row_weight, float *nll, float *lse, int32_t *status, float *loss,
               void *grad_hidden, void *grad_weight, void *workspace, size_t workspace_bytes, void *stream);

/* topk_val [N, 32], topk_idx [N, 32], row_sample [N], rewards [S], kl [N],
 * row_weight_out [N] or NULL, status [N] or NULL as in sv_kd; the rest as above. */
int sv_head_kd(const sv_head_shape_t *shape, const void *hidden, const float *hidden_scale, const void *weight,
               const float *topk_val, const int32_t *topk_idx, const int32_t *row_sample, const float *rewards,
               float *kl, float *row_weight_out, int32_t *status, float *loss, void *grad_hidden, void *grad_weight,
               void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SV_HEAD_H */
