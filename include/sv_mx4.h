/*
 * sv_mx4.h -- C ABI of microscaled 4-bit rows and of a vocabulary head held in them, for
 * AMD MI355X (gfx950).  Same library (libspec_verify.so).
 *
 *   sv_mx4_pack / sv_mx4_unpack  rows in 4 bits, 32 elements to a power-of-two scale
 *   sv_head_logits4              logits of hidden rows under a head held so
 *
 * The head of a drafter is what this is for: verification keeps the rollout's
 * distribution whatever the drafter's is (ReSpec notes, "2 . background"), so its head may
 * be coarse, and at a quarter of the bytes a decode step of it takes a quarter of the time.
 *
 * All calls enqueue on `stream` (a hipStream_t; NULL = default stream) and return without
 * synchronising; they allocate nothing and keep no state between calls, so they can be
 * captured in HIP graphs.  Argument errors return a negative SV_ERR_* code (spec_verify.h)
 * before anything is enqueued.  Results are deterministic: every sum runs in a fixed order.
 * Device pointers are caller-owned and on the current device.  A workspace is scratch memory
 * of at least the *_workspace_bytes of the shape, 256-byte aligned, with any contents, before
 * and after; calls that share one must not overlap in time.
 */
#ifndef SV_MX4_H
#define SV_MX4_H

#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"
#include "sv_head.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element type of rows held as 4-bit codes with a scale per 32 elements (beside SV_F32,
 * SV_BF16 and SV_I8) */
#define SV_MX4 3

/* elements that share a scale */
#define SV_MX4_BLOCK 32

/* ---------------------------------------------------------------- 4-bit rows
 * The OCP microscaling format MXFP4.  A code is a sign (bit 3) and one of 0, 1/2, 1, 3/2,
 * 2, 3, 4, 6 (bits 0 to 2); byte j of a row holds element 2 j in its low half and 2 j + 1 in
 * its high half.  A scale byte e stands for 2^(e - 127), 255 for NaN.
 *
 * For each block b of 32 elements (a row's last may be shorter):
 *   e = max(floor(log2(max_k |x_k|)) - 2 + 127, 0), 0 for a block of zeros
 *   code_k = x_k / 2^(e - 127) to the nearest code, ties to the one with bit 0 clear,
 *            magnitudes above 6 (below 8) to 6
 *   unpacked y_k = code_k 2^(e - 127)
 * Both divisions and products are exact.  A block holding a NaN or an infinity gets scale
 * 255 and codes 0 (unpacked: NaN).  Unpacked values beyond the type's range (scales above
 * 252, which pack does not make) are infinite.
 * x [N, H] (SV_F32 or SV_BF16) with row stride x_stride elements, codes [N, (H + 1) / 2] with
 * row stride codes_stride bytes, scale [N, (H + 31) / 32] with row stride scale_stride bytes, y
 * [N, H] contiguous in y_dtype; a stride of 0 means no gaps.  The last byte's high half is 0
 * where H is odd.  Bytes between a row's end and a stride are not written.
 * N = 0: returns SV_OK and enqueues nothing.
 */
int sv_mx4_pack(int32_t N, int32_t H, int32_t dtype, const void *x, int64_t x_stride, uint8_t *codes,
                int64_t codes_stride, uint8_t *scale, int64_t scale_stride, void *stream);
int sv_mx4_unpack(int32_t N, int32_t H, const uint8_t *codes, int64_t codes_stride, const uint8_t *scale,
                  int64_t scale_stride, int32_t y_dtype, void *y, void *stream);

/* ------------------------------------------------------------ 4-bit head logits
 *   logits[n,v] = sum_k x~[n,k] w~[v,k]
 * over the values that the codes and scales stand for, summed in fp32 and rounded to the
 * output's type once.  x~ is either given (hidden_dtype SV_MX4, with hidden_scale) or formed
 * from fp32 or bf16 rows as sv_mx4_pack does.  A block whose scale is NaN makes its row's (a
 * weight block: its column's) logits NaN, which spec_verify reports.
 */
typedef struct {
    int32_t N;                    /* hidden rows, >= 0 (0: nothing to do) */
    int32_t H;                    /* hidden width, 1 .. SV_HEAD_MAX_H */
    int32_t V;                    /* vocabulary entries, 1 .. SV_HEAD_MAX_V */
    int32_t hidden_dtype;         /* SV_F32, SV_BF16 or SV_MX4 */
    int32_t out_dtype;            /* SV_F32 or SV_BF16 */
    int64_t hidden_stride;        /* between hidden rows: elements, SV_MX4: bytes; 0: no gaps */
    int64_t hidden_scale_stride;  /* bytes between hidden scale rows (SV_MX4); 0: no gaps */
    int64_t weight_stride;        /* bytes between weight code rows; 0: no gaps */
    int64_t weight_scale_stride;  /* bytes between weight scale rows; 0: no gaps */
    int64_t out_stride;           /* elements between logits rows; 0 means V */
} sv_logits4_shape_t;

size_t sv_head_logits4_workspace_bytes(const sv_logits4_shape_t *shape);

/* hidden [N, H]; hidden_scale (SV_MX4 only, else ignored); weight_codes [V, (H + 1) / 2] and
 * weight_scale [V, (H + 31) / 32]; logits [N, V] (out_dtype). */
int sv_head_logits4(const sv_logits4_shape_t *shape, const void *hidden, const uint8_t *hidden_scale,
                    const uint8_t *weight_codes, const uint8_t *weight_scale, void *logits, void *workspace,
                    size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SV_MX4_H */
