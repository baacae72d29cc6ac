/*
 * fp8bs_layer.h - the entry points of libfp8bs.so that stand between the products
 * of a transformer block: gradient norms and clipping.
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
 *   counts n numbers of values, >= 0 and at most 2^40
 *   types  n types, FP8BS_F32 or FP8BS_BF16 (else FP8BS_EINVAL)
 *   n      0 .. FP8BS_MAX_TENSORS (else FP8BS_EINVAL); without values the norm is 0
 *   norm   one fp32 on the device, out
 *   workspace of fp8bs_grad_norm_workspace(n) bytes (else FP8BS_EINVAL)
 */
int64_t fp8bs_grad_norm_workspace(int32_t n);
fp8bs_status fp8bs_grad_norm(const void* const* grads, const int64_t* counts, const int32_t* types, int32_t n,
                             float* norm, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * fp8bs_clip_grads - out = g * min(1, max_norm / (norm + eps)), each product
 *   rounded once to g's type, from a norm that is on the device (fp8bs_grad_norm's, or
 *   one that several processes have joined).
 *   outs   n device pointers of g's types and counts.  outs[i] is grads[i] (in
 *          place; a factor of 1 then writes nothing) or overlaps no tensor of the call;
 *          tensors that are written overlap no other one (else FP8BS_EINVAL)
 *   norm   one fp32 on the device.  An infinite norm makes the factor 0, a NaN makes
 *          it NaN, as the formula has it.
 *   max_norm, eps  finite, >= 0 (else FP8BS_EINVAL)
 */
fp8bs_status fp8bs_clip_grads(const void* const* grads, void* const* outs, const int64_t* counts,
                              const int32_t* types, int32_t n, const float* norm, double max_norm, double eps,
                              void* stream);

/*
 * fp8bs_clip_grad_norm - both: the norm, out as by fp8bs_grad_norm, and the clipping
 *   with that norm before it is rounded to fp32.  workspace as for fp8bs_grad_norm.
 */
fp8bs_status fp8bs_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* counts,
                                  const int32_t* types, int32_t n, double max_norm, double eps, float* norm,
                                  void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BS_LAYER_H */
