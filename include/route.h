/*
 * route.h -- C ABI of what stands round the product grouped by expert
 * (fp8_grouped_gemm) of the MI355X (gfx950) library: the router ahead of it (the
 * choice of experts, their counts, the order of the rows, the balance loss and its
 * gradient) and the weighted sum of the experts' rows behind it with its gradient.
 * Same shared library and status codes as w4a16.h.
 *
 * For token t with logits l: p = softmax(l) over the E experts; chosen are the `top`
 * largest logits, the lowest index first among equal ones.  An expert whose logit is
 * -infinity or NaN is never chosen: a token with fewer others has slots without an
 * expert.  A token that valid marks with 0 (padding behind a sequence) has none at all
 * and counts nowhere.  With ROUTE_RENORMALIZE the weights of a token's chosen experts
 * are p divided by their sum, otherwise p itself.
 *
 *   balance loss  L = sum over e of pull[e] * sum over valid t of p[t][e],
 *   pull[e] = E * counts[e] / (V * top) / V,  V the number of valid tokens
 *
 * (E times the sum of each expert's share of the slots times its mean probability: 1
 * when all are used alike); 0 when V is 0.  pull is a constant to the gradient.
 *
 * A NaN or +infinity among a token's logits makes its probabilities NaN: its weights,
 * the loss and its gradients show it, its experts and the order stay in range.  Logits
 * that are all -infinity give probabilities 0.  Sums are fp32 in a fixed order (that of a
 * token's chosen probabilities, which RENORMALIZE divides by, is kept in steps of 2^-26 at
 * most of its largest): equal calls give equal bits, and a token's experts and weights do
 * not depend on the other tokens.
 *
 * Conventions are those of w4a16.h (plain C types, caller-owned device pointers, stream
 * as void*, asynchronous, nothing allocated, every argument validated on the host before
 * any HIP call); pointers need the alignment of their elements (valid: a byte's).  1 <= E
 * <= ROUTE_MAX_EXPERTS, 1 <= top <= min(E, ROUTE_MAX_TOP) (beyond the maxima:
 * W4A16_ERR_UNSUPPORTED), T < 2^26, T * top < 2^31, T * ld < 2^40.
 */
#ifndef ROUTE_H
#define ROUTE_H

#include <stddef.h>
#include <stdint.h>

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of the logits (route_tokens*) or rows (route_combine*: not FP32). */
#define ROUTE_FP16 0x0u
#define ROUTE_BF16 0x1u
#define ROUTE_FP32 0x2u
#define ROUTE_TYPE_MASK 0x3u
#define ROUTE_RENORMALIZE 0x10u

#define ROUTE_MAX_EXPERTS 1024
#define ROUTE_MAX_TOP 32

/* Workspace bytes route_tokens needs (0 = none, also if the arguments are bad).  It is
 * laid out like the workspaces of w4a16_gemm, whose counters it leaves as they are, and
 * needs no fill of its own.  The call is several launches that hand on through it what
 * they found: until the last of them has run, no other call may use it, also not one that
 * another host thread launches on the same stream (it could come between them). */
size_t route_workspace_bytes(int64_t T, int64_t E, int64_t top);

/*
 *   logits   dev, [T] rows of E elements, ld apart;  valid  dev, uint8 [T], or NULL
 *            (every token is real);
 *   weights  dev, float [T][top];  experts  dev, int32 [T][top], -1 where there is none;
 *   counts   dev, int32 [E]: slots of each expert;
 *   offsets  dev, int32 [E+1]: rows offsets[e] .. offsets[e+1]-1 are expert e's;
 *   rows     dev, int32 [T*top]: the token of each row, an expert's in the order of the
 *            tokens, -1 behind offsets[E]: the `rows` of fp8_grouped_gemm;
 *   places   dev, int32 [T][top]: the row of each slot, -1 where there is none;
 *   loss     dev, float [1], and pull  dev, float [E]: the balance loss, both NULL if it
 *            is not wanted.
 * T = 0 is a call like any other (counts, offsets and loss are zeros).
 */
w4a16_status_t route_tokens(const void *logits, int64_t ld, const uint8_t *valid, float *weights,
                            int32_t *experts, int32_t *counts, int32_t *offsets, int32_t *rows,
                            int32_t *places, float *loss, float *pull, int64_t T, int64_t E,
                            int64_t top, uint32_t flags, void *workspace, size_t workspace_bytes,
                            void *stream);

/*
 * dlogits, in the logits' type, contiguous [T][E]: the gradient of what dweights [T][top]
 * (fp32, NULL: zeros) and dloss (dev, float [1], NULL: zero) pull at.  logits, ld, valid
 * and flags as given to route_tokens, weights, experts and pull as it left them (pull
 * may be NULL without dloss).
 *   a = dweights, w = weights:
 *   d[i]   = p[i] * (dloss * (pull[i] - sum over e of p[e] pull[e]))
 *   d[i]  += p[i] * ((a of i if chosen, else 0) - sum over j of a[j] w[j])     plain
 *   d[ej] += w[j] * (a[j] - sum over j of a[j] w[j])                           RENORMALIZE
 * Rows of tokens that are not valid are zeros.  T = 0 is a call without work.
 */
w4a16_status_t route_tokens_backward(const void *logits, int64_t ld, const uint8_t *valid,
                                     const float *weights, const int32_t *experts,
                                     const float *pull, const float *dweights, const float *dloss,
                                     void *dlogits, int64_t T, int64_t E, int64_t top,
                                     uint32_t flags, void *stream);

/*
 * out[t] = residual[t] + sum over j of weights[t][j] * y[places[t][j]], summed in fp32 in
 * the order of j and rounded once.  A place outside [0, R) adds nothing, whatever its
 * weight.
 *   y        dev, fp16 or bf16 [R] rows of N elements, ldy apart;
 *   weights  dev, float [T][top];  places  dev, int32 [T][top];
 *   residual dev, [T] rows of N, ldr apart, or NULL;  out  dev, [T][N] contiguous (it may
 *            be residual if that is contiguous).
 * N >= 1 and below 2^24; rows may start at any element.
 */
w4a16_status_t route_combine(const void *y, int64_t ldy, const float *weights,
                             const int32_t *places, const void *residual, int64_t ldr, void *out,
                             int64_t T, int64_t R, int64_t N, int64_t top, uint32_t flags,
                             void *stream);

/*
 * dy[places[t][j]] = weights[t][j] * dout[t], rounded once, and dweights[t][j] = the inner
 * product of dout[t] and y[places[t][j]] in fp32 (0 for a place outside [0, R)).  Places
 * inside must differ.
 *   dout     dev, [T] rows of N, ldd apart;  y, ldy, weights, places as above;
 *   routed   dev, int32 [1] (offsets + E), or NULL: rows of dy from routed[0] on are
 *            zeros, and a place there is like one outside; rows before it (without it:
 *            all rows) that no place names are not written;
 *   dy       dev, [R][N] contiguous;  dweights  dev, float [T][top].
 */
w4a16_status_t route_combine_backward(const void *dout, int64_t ldd, const void *y, int64_t ldy,
                                      const float *weights, const int32_t *places,
                                      const int32_t *routed, void *dy, float *dweights, int64_t T,
                                      int64_t R, int64_t N, int64_t top, uint32_t flags,
                                      void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ROUTE_H */
