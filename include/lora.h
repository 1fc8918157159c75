/*
 * lora.h -- C ABI of the low-rank adapters of many requests beside a projection
 * that all of them share, of the MI355X (gfx950) library.  Same shared library and
 * status codes as w4a16.h.
 *
 *   out[m] = RNE_out( base[m] + (scale[a] * (x[m] . A[a]^T)) . B[a]^T ),  a = ids[m]
 *
 * base is what the shared projection (w4a16_gemm, fp8_gemm, ...) gave for x.  A row whose
 * id is outside [0, L) has no adapter: out[m] = base[m], bit for bit.  The rows of an
 * adapter may lie anywhere; what an adapter or a row holds (NaN and infinities too) is
 * seen in that adapter's or row's outputs only (an infinity in B as an infinity or a NaN,
 * since a part of what it is multiplied by may be 0).  The R inner products with A are kept in
 * fp32; as operand of the second product each is the sum of numbers of the activations'
 * type: bf16 of three, which hold all its 24 bits, fp16 of two, which hold 22 (after a row's
 * finite ones were brought near 2^14 by a power of two).  Sums have a fixed order: equal
 * calls give equal bits, and a row's result does not depend on the other rows' ids.
 *
 * Conventions are those of w4a16.h (plain C types, caller-owned device pointers, stream
 * as void*, asynchronous, nothing allocated, every argument validated on the host before
 * any HIP call).  R % 8 == 0 and R <= LORA_MAX_RANK (a smaller adapter is filled up with
 * zeros), K % 8 == 0 (rows of E4M3: K % 16 == 0), otherwise W4A16_ERR_UNSUPPORTED; any N;
 * N, K, M, L < 2^24, M * N < 2^37.  x, a and b are 16-byte aligned, row strides (in elements)
 * of x multiples of 16 bytes; base and out may start at any element.
 */
#ifndef LORA_H
#define LORA_H

#include <stddef.h>
#include <stdint.h>

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of a, b, base and out, and of x unless LORA_X_FP8. */
#define LORA_FP16 0x0u
#define LORA_BF16 0x1u
/* x holds E4M3 codes with a scale per row and 128 columns (the rows of fp8_gemm). */
#define LORA_X_FP8 0x10u

#define LORA_MAX_RANK 256

/* Workspace bytes lora_add needs (0 if the arguments are bad or M is 0).  It is laid out
 * like the workspaces of w4a16_gemm, whose counters it leaves as they are, and needs no
 * fill of its own.  The call is several launches that hand on through it what they found:
 * until the last of them has run, no other call may use it, also not one that another host
 * thread launches on the same stream (it could come between them). */
size_t lora_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L,
                            uint32_t flags);

/*
 *   base   dev, [M] rows of N, ldb apart;
 *   x      dev, [M] rows of K, ldx apart;  xs  dev, float [M][ceil(K/128)] with
 *          LORA_X_FP8, otherwise NULL;
 *   a      dev, [L][R][K];  b  dev, [L][N][R];  scale  dev, float [L], or NULL (ones);
 *   ids    dev, int32 [M];
 *   out    dev, [M] rows of N, ldo apart: base itself (with ldo = ldb; rows without an
 *          adapter are not touched then) or memory that overlaps none of the inputs.
 */
w4a16_status_t lora_add(const void *base, int64_t ldb, const void *x, int64_t ldx,
                        const float *xs, const void *a, const void *b, const float *scale,
                        const int32_t *ids, void *out, int64_t ldo, int64_t M, int64_t N,
                        int64_t K, int64_t R, int64_t L, uint32_t flags, void *workspace,
                        size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_H */
