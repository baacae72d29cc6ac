// Internal launcher declarations of the operators between the products (include/fp8bs_layer.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bs {
// What a product's epilogue does: z = acc + bias, C = act(z) + residual, pre = z; any of the
// pointers may be null.
struct Epilogue {
  const uint16_t *bias, *residual;
  uint16_t* pre;
  int act;  // an Activation
};
hipError_t launch_gemm_g128_epilogue(const void* a, const float* sa, const void* bt, const float* sbt,
                                     const Epilogue& e, void* c, int64_t M, int64_t N, int64_t K,
                                     hipStream_t stream);
int64_t epilogue_backward_workspace(int64_t rows, int64_t n);
// z may be null with ACT_NONE; dz and dbias (and then workspace) may be null
hipError_t launch_epilogue_backward(const void* dout, const void* z, int act, int64_t rows, int64_t n, void* dz,
                                    void* q, float* scales, float* dbias, bool accumulate, float* workspace,
                                    hipStream_t stream);
// q and scales, y, h, residual, beta, mean and rstd may be null
hipError_t launch_layernorm(const void* x, const void* residual, const void* gamma, const void* beta, float eps,
                            int64_t rows, int64_t d, void* h, void* q, float* scales, void* y, float* mean,
                            float* rstd, hipStream_t stream);
int layernorm_max_cols();
int64_t layernorm_backward_workspace(int64_t rows, int64_t d);
hipError_t launch_layernorm_backward(const void* dy, const void* h, const void* gamma, const float* mean,
                                     const float* rstd, const void* dresidual, int64_t rows, int64_t d, void* dx,
                                     float* dgamma, float* dbeta, bool accumulate, float* workspace,
                                     hipStream_t stream);
hipError_t set_layernorm_attributes();
int64_t moe_decode_workspace(int tokens, int top, int experts, int64_t hidden, int64_t inner);
hipError_t launch_moe_decode(const void* x, const int32_t* ids, const float* weights, const void* w1,
                             const float* s1, const void* w2, const float* s2, const void* residual, void* out,
                             int tokens, int top, int experts, int64_t hidden, int64_t inner, void* workspace,
                             hipStream_t stream);
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
