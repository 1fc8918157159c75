/*
 * rowquant.h -- C ABI of the fused producers of quantised rows of the MI355X
 * (gfx950) library: the RMS norm (with the residual's addition) and the gated
 * activation, each ending in the rows that the library's products read.  Same
 * shared library and status codes as w4a16.h.
 *
 * Kinds of output, v being the fp32 value of an element:
 *   ROWQUANT_FP8   q uint8 [T][W] E4M3, s float [T][ceil(W/128)]: with a the
 *                  block's largest |v| or 2^-110 if that is smaller,
 *                  s = a / 448 and q = E4M3(v * (448 / a)); for fp8_gemm.
 *   ROWQUANT_INT8  q int8 [T][W], s float [T]: s = max |v| / 127 of the row,
 *                  q = round-half-even(v / s); a row of zeros gives zeros; for
 *                  w4a8_gemm.
 *   ROWQUANT_MX    q uint8 [T][W] E4M3, s uint8 [T][W/32] E8M0, the rule of
 *                  mxfp4_quantize_rows; for mxfp4_gemm.
 *   ROWQUANT_X16   q in the inputs' dtype [T][W], s NULL; for w4a16_gemm.
 * Roundings to E4M3 are to the nearest value, ties to the even code,
 * saturating at 448.  A v that is NaN or infinite (an input that is, or a result
 * beyond fp32) shows: in its element (X16), as a NaN or infinite scale of its block
 * (FP8) or row (INT8), as the scale 0xFF, the E8M0 NaN (MX); such a block's or row's
 * codes mean nothing.  Other blocks and rows are as without it, except that one such
 * input of the norm is in its whole row's mean.
 *
 * Conventions are those of w4a16.h, but s needs the alignment of its elements
 * only.  W % 16 == 0 (MX: W % 32 == 0), otherwise
 * W4A16_ERR_UNSUPPORTED; row strides (in elements) are multiples of 8 and at
 * least W; T < 2^31.  T = 0 is a call without work.
 */
#ifndef ROWQUANT_H
#define ROWQUANT_H

#include <stddef.h>
#include <stdint.h>

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Flags: the inputs' dtype and the kind of output. */
#define ROWQUANT_IN_FP16 0x0u
#define ROWQUANT_IN_BF16 0x1u
#define ROWQUANT_FP8  0x00u
#define ROWQUANT_INT8 0x10u
#define ROWQUANT_MX   0x20u
#define ROWQUANT_X16  0x30u
#define ROWQUANT_KIND_MASK 0x30u

#define ROWQUANT_MAX_ROW 131072   /* widest row of the norm and of the int8 kind */

/*
 * h = x + residual (x alone if residual is NULL), kept in fp32;
 * v = h * (1 / sqrt(mean(h^2) + eps)) * weight; q, s of v.
 *   x         dev, [T] rows of W elements, ldx apart;  residual the same with ldr;
 *   weight    dev, [W];  h_out  dev, [T][W] in the inputs' dtype, h rounded once
 *             (NULL: not wanted; it may be x or residual if those are contiguous).
 *   W <= ROWQUANT_MAX_ROW, eps >= 0 (with eps = 0 a row of zeros has no norm).
 */
w4a16_status_t rowquant_rmsnorm(const void *x, int64_t ldx, const void *residual, int64_t ldr,
                                const void *weight, float eps, void *h_out, void *q, void *s,
                                int64_t T, int64_t W, uint32_t flags, void *stream);

/*
 * v = gate / (1 + exp(-gate)) * up; q, s of v.  ROWQUANT_INT8: W <=
 * ROWQUANT_MAX_ROW; the other kinds take any W < 2^31.
 *   gate, up  dev, [T] rows of W elements, ldg and ldu apart (the halves of one
 *             [T][2W] tensor, for instance).
 */
w4a16_status_t rowquant_swiglu(const void *gate, int64_t ldg, const void *up, int64_t ldu, void *q,
                               void *s, int64_t T, int64_t W, uint32_t flags, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ROWQUANT_H */
