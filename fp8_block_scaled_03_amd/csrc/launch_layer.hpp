// Internal launcher declarations of the operators between the products (include/fp8bs_layer.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bs {
// The gradients of one call, on the host.
struct Grads {
  const void* const* src;
  void* const* dst;  // null for the norm alone
  const int64_t* counts;
  const int32_t* types;
  int n;
};
int64_t grad_norm_workspace(int n);
// norm alone: `norm` out.
hipError_t launch_grad_norm(const Grads& g, float* norm, double* workspace, hipStream_t stream);
// workspace null: clipping by the norm at `norm`; else the norm first, out at `norm`.
hipError_t launch_clip_grads(const Grads& g, double max_norm, double eps, float* norm, double* workspace,
                             hipStream_t stream);
}  // namespace fp8bs
