/*
 * fp8bs_layer.h - the entry points of libfp8bs.so that stand between the products
 * of a transformer block: layer norm with its backward pass, products with bias,
 * activation and residual in their epilogue and its backward pass, a whole
 * mixture-of-experts layer for a few tokens, gradient norms and clipping.
 * Status codes, pointer ownership, streams and errors are those of fp8bs.h; the
 * E4M3 format and the quantizer's rule for 128 values are those of fp8bs_g128.h.
 *
 * Conventions of this header
 *   - The library allocates nothing.  An entry point that needs memory for partial
 *     sums takes a workspace (device memory, 16-byte aligned) of at least the size
 *     that its ..._workspace function returns for the same sizes; its contents
 *     need not be set and mean nothing afterwards.  It is in use from the call until
 *     the stream has passed it: calls on different streams, and graphs that may
 *     be replayed at the same time, each need one of their own.
 *   - Results do not depend on timing: every sum has a fixed order.
 */
#ifndef FP8BS_LAYER_H
#define FP8BS_LAYER_H

#include "fp8bs.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fp8bs_layernorm_quantize_tg128 - residual add + layer norm + the row quantizer of
 *   128 values, in one pass over each row:
 *     residual != NULL:  h = bf16(x + residual) (nearest even), written to h if given
 *     residual == NULL:  h = x (and the argument h is not used)
 *     mean = sum(h) / d,  var = sum((h - mean)^2) / d,  rstd = 1 / sqrt(var + eps)  (fp32)
 *     y_i = (h_i - mean) * rstd * gamma_i + beta_i                                (fp32)
 *     q, scales = the quantizer's rule of fp8bs_g128.h on the fp32 y (128 columns each)
 *   x [rows, d] bf16, residual [rows, d] bf16 or NULL, gamma [d] bf16,
 *   beta [d] bf16 or NULL (no bias)
 *   h [rows, d] bf16 out or NULL; may be residual or x themselves (in place)
 *   q [rows, d] E4M3 out, scales [rows, ceil128(d)] fp32 out
 *   y [rows, d] bf16 out (rounded to nearest) or NULL
 *   mean, rstd [rows] fp32 out for the backward pass, or both NULL
 *   eps finite and >= 0 (else FP8BS_EINVAL); with eps == 0 a row of equal values has
 *   no defined result.  d % 16 == 0, d <= 16384, rows <= 2^30 (else FP8BS_ESHAPE);
 *   rows == 0 or d == 0: no-op.  Matrices, gamma and beta are 16-byte aligned, scales
 *   and statistics 4-byte (else FP8BS_EALIGN).  A row's results depend on that row
 *   only.  The sums are fp32 ones: a row whose values, or whose squared deviations from
 *   the mean, add up to 2^128 or more is beyond their range (deviations of 2^57 throughout a
 *   row of 16384, of 2^62 throughout one of 16), and with an eps next to 0 deviations below
 *   2^-63 lose digits.  Outputs other than h overlap no input, and none another one.
 */
fp8bs_status fp8bs_layernorm_quantize_tg128(const void* x_bf16, const void* residual_bf16, const void* gamma_bf16,
                                            const void* beta_bf16, float eps, int64_t rows, int64_t d, void* h_bf16,
                                            void* q_e4m3, float* scales, void* y_bf16, float* mean, float* rstd,
                                            void* stream);

/* fp8bs_layernorm - the same without codes; y is required. */
fp8bs_status fp8bs_layernorm(const void* x_bf16, const void* residual_bf16, const void* gamma_bf16,
                             const void* beta_bf16, float eps, int64_t rows, int64_t d, void* h_bf16, void* y_bf16,
                             float* mean, float* rstd, void* stream);

/*
 * fp8bs_layernorm_backward - the gradients of y = (h - mean) rstd gamma + beta, with
 *   xh = (h - mean) * rstd and g = dy * gamma, all in fp32:
 *     dx     = rstd * (g - sum(g)/d - xh * sum(g xh)/d) (+ dresidual), rounded to bf16
 *     dgamma = sum over the rows of dy * xh,  dbeta = sum over the rows of dy
 *   dy, h [rows, d] bf16, gamma [d] bf16, mean, rstd [rows] fp32 (the forward call's)
 *   dresidual [rows, d] bf16 or NULL: the gradient that reaches h past the norm
 *   dx [rows, d] bf16 out
 *   dgamma, dbeta [d] fp32 out, each or NULL; if accumulate != 0 the sums are added
 *      to what they hold.  rows == 0: zeros (or nothing is added).
 *   workspace of fp8bs_layernorm_backward_workspace(rows, d) bytes (else FP8BS_EINVAL).
 *   Sizes and alignment as above; outputs overlap no input.
 */
int64_t fp8bs_layernorm_backward_workspace(int64_t rows, int64_t d);
fp8bs_status fp8bs_layernorm_backward(const void* dy_bf16, const void* h_bf16, const void* gamma_bf16,
                                      const float* mean, const float* rstd, const void* dresidual_bf16, int64_t rows,
                                      int64_t d, void* dx_bf16, float* dgamma, float* dbeta, int32_t accumulate,
                                      void* workspace, int64_t workspace_bytes, void* stream);

/* Activations of an epilogue. */
#define FP8BS_ACT_NONE 0
#define FP8BS_ACT_RELU 1
#define FP8BS_ACT_GELU 2      /* z Phi(z), Phi the normal distribution's function  */
#define FP8BS_ACT_GELU_TANH 3 /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2   */
#define FP8BS_ACT_SILU 4      /* z / (1 + exp(-z))                                 */

/*
 * fp8bs_gemm_tg128_nt_epilogue - fp8bs_gemm_tg128_nt with an epilogue on its fp32
 *   accumulators, before the one rounding of the result:
 *     z = A Bt' + bias,  c = bf16(act(z) + residual),  pre = bf16(z)
 *   a, sa, bt, sbt, M, N, K as for fp8bs_gemm_tg128_nt; K == 0: the product is 0
 *   bias [N] bf16 or NULL, activation one of FP8BS_ACT_* (else FP8BS_EINVAL)
 *   residual [M, N] bf16 or NULL; may be c itself (in place)
 *   c [M, N] bf16 out; pre [M, N] bf16 out or NULL, apart from the other arguments
 *      (c or residual itself: FP8BS_EINVAL)
 *   The activation is fp32 arithmetic, off by at most 2^-15 of its result, whose
 *   magnitudes below 2^-118 may come out as 0; an exact zero is stored as +0.  At z = -inf
 *   gelu is 0, its limit; gelu_tanh and silu are NaN, as their formulas have it.
 *   Results are batch invariant as fp8bs_gemm_tg128_nt's.
 */
fp8bs_status fp8bs_gemm_tg128_nt_epilogue(const void* a, const float* sa, const void* bt, const float* sbt,
                                          const void* bias_bf16, int32_t activation, const void* residual_bf16,
                                          void* c_bf16, void* pre_bf16, int64_t M, int64_t N, int64_t K, void* stream);

/*
 * fp8bs_epilogue_backward_quantize_tg128 - the gradient of act(z) + residual with
 *   respect to z (the residual's is dout itself), with the quantizer that the input
 *   gradient's product needs and the gradient of the bias:
 *     dz     = dout * act'(pre)  (fp32), rounded to bf16 (for the weight gradient)
 *     q, scales = the row quantizer's rule of fp8bs_g128.h on the fp32 dz
 *     dbias  = sum over the rows of the fp32 dz
 *   relu's derivative at 0 is 0, a derivative at an infinite z its limit.
 *   dout [rows, n] bf16, pre [rows, n] bf16 (the forward call's; with FP8BS_ACT_NONE
 *   it is not read and may be NULL), dz [rows, n] bf16 out or NULL, q [rows, n] E4M3
 *   out, scales [rows, ceil128(n)] fp32 out
 *   dbias [n] fp32 out or NULL; if accumulate != 0 the sums are added to what it holds.
 *      rows == 0: zeros (or nothing is added).
 *   workspace of fp8bs_epilogue_backward_workspace(rows, n) bytes (else
 *   FP8BS_EINVAL); not used without dbias.
 *   n % 16 == 0, rows and n at most 2^30 (else FP8BS_ESHAPE); n == 0: no-op.
 *   Outputs overlap no input, and none another one.
 */
int64_t fp8bs_epilogue_backward_workspace(int64_t rows, int64_t n);
fp8bs_status fp8bs_epilogue_backward_quantize_tg128(const void* dout_bf16, const void* pre_bf16, int32_t activation,
                                                    int64_t rows, int64_t n, void* dz_bf16, void* q_e4m3,
                                                    float* scales, float* dbias, int32_t accumulate, void* workspace,
                                                    int64_t workspace_bytes, void* stream);

/* Most choices (tokens * top) of fp8bs_moe_decode_b128. */
#define FP8BS_MAX_MOE_CHOICES 512

/*
 * fp8bs_moe_decode_b128 - a whole mixture-of-experts layer for a few tokens: per
 *   token t, with e = ids[t,j] for its choices j = 0 .. top-1,
 *     [g | u] = W1[e] x[t],  y = silu(g) * u,
 *     out[t]  = bf16(sum_j weights[t,j] * W2[e] y (+ residual[t]))
 *   The weights are E4M3 codes with a scale per 128x128 block (fp8bs_quantize_b128);
 *   x is bf16 and is not quantized, [g | u] is fp32 and y is held to 2^-17 of itself.
 *   Products are exact, sums fp32; the choices are added in order.
 *   x [tokens, hidden] bf16
 *   ids [tokens, top] int32 on the device, read when the kernels run, so a captured graph
 *      follows them.  A choice whose id is outside [0, experts) adds nothing
 *      (an expert that another process holds, a token that pads a batch).  A
 *      token may name an expert more than once.
 *   weights [tokens, top] fp32; those of skipped choices are not used
 *   w1 [experts, 2 inner, hidden] E4M3 (inner gates, then inner ups),
 *   s1 [experts, ceil128(2 inner), ceil128(hidden)] fp32
 *   w2 [experts, hidden, inner] E4M3, s2 [experts, ceil128(hidden), ceil128(inner)] fp32
 *   residual [tokens, hidden] bf16 or NULL; may be out itself (in place)
 *   out [tokens, hidden] bf16 out, apart from the other arguments
 *   1 <= top and 1 <= experts <= FP8BS_MAX_GROUPS (else FP8BS_EINVAL);
 *   tokens * top <= FP8BS_MAX_MOE_CHOICES, hidden and inner multiples of 16, hidden <=
 *   32768, 16 <= inner <= 32768 (else FP8BS_ESHAPE); tokens == 0 or hidden == 0: no-op.
 *   workspace of fp8bs_moe_decode_b128_workspace(...) bytes (else FP8BS_EINVAL).
 *   Results are batch invariant: a token's depend on that token only.
 *   For few choices of an expert: from about 15 of each on, the products of quantized
 *   activations (fp8bs_grouped_gemm_tg128_nt) take less time, with the codes of x and y
 *   as the price.
 */
int64_t fp8bs_moe_decode_b128_workspace(int64_t tokens, int64_t top, int64_t experts, int64_t hidden,
                                        int64_t inner);
fp8bs_status fp8bs_moe_decode_b128(const void* x_bf16, const int32_t* ids_dev, const float* weights, const void* w1,
                                   const float* s1, const void* w2, const float* s2, const void* residual_bf16,
                                   void* out_bf16, int64_t tokens, int64_t top, int64_t experts, int64_t hidden,
                                   int64_t inner, void* workspace, int64_t workspace_bytes, void* stream);

/* Types of a gradient. */
#define FP8BS_F32 0
#define FP8BS_BF16 1

/* Most tensors of one call. */
#define FP8BS_MAX_TENSORS 65536

/*
 * fp8bs_grad_norm - norm = sqrt(sum over all tensors and values of g^2), as fp32.
 *   Squares and sums are held in 64 bits, so neither large nor small values are
 *   lost; an infinity gives an infinite norm, a NaN a NaN.
 *   grads  n device pointers, in a host array that is read before the call returns
 *          (so are the next two); each aligned to its type, NULL where the count is 0
 *   counts n numbers of values, >= 0 (else FP8BS_EINVAL) and at most 2^36 (else FP8BS_ESHAPE)
 *   types  n types, FP8BS_F32 or FP8BS_BF16 (else FP8BS_EINVAL)
 *   n      0 .. FP8BS_MAX_TENSORS (else FP8BS_EINVAL); without values the norm is 0
 *   norm   one fp32 on the device, out
 *   workspace of fp8bs_grad_norm_workspace(n) bytes (else FP8BS_EINVAL)
 */
int64_t fp8bs_grad_norm_workspace(int32_t n);
fp8bs_status fp8bs_grad_norm(const void* const* grads, const int64_t* counts, const int32_t* types, int32_t n,
                             float* norm, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * fp8bs_clip_grads - out = g * min(1, max_norm / (norm + eps)), the factor rounded to
 *   fp32, each product to fp32 and from there to g's type, from a norm that is on the device (fp8bs_grad_norm's, or
 *   one that several processes have joined).
 *   outs   n device pointers of g's types and counts.  outs[i] is grads[i] (in
 *          place; a factor of 1 then writes nothing) or overlaps no tensor of the call;
 *          tensors that are written overlap no other one, and norm none (else FP8BS_EINVAL)
 *   norm   one fp32 on the device.  An infinite norm makes the factor 0, a NaN makes
 *          it NaN, as the formula has it.
 *   max_norm, eps  finite, >= 0 (else FP8BS_EINVAL)
 */
fp8bs_status fp8bs_clip_grads(const void* const* grads, void* const* outs, const int64_t* counts,
                              const int32_t* types, int32_t n, const float* norm, double max_norm, double eps,
                              void* stream);

/*
 * fp8bs_clip_grad_norm - both: the norm, out as by fp8bs_grad_norm, and the clipping
 *   with that norm before it is rounded to fp32.  norm overlaps no tensor of the call (else
 *   FP8BS_EINVAL); workspace as for fp8bs_grad_norm.
 */
fp8bs_status fp8bs_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* counts,
                                  const int32_t* types, int32_t n, double max_norm, double eps, float* norm,
                                  void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BS_LAYER_H */
