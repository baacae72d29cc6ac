// C ABI of the operators between the products (see include/fp8bs_layer.h).
// Host-side argument checks, then the launches on the caller's stream.
#include "fp8bs_layer.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <vector>

#include "launch_layer.hpp"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// hipErrorNotSupported from a launcher: the grid would be too large
fp8bs_status from_launch(hipError_t e) {
  if (e == hipErrorNotSupported) return FP8BS_ESHAPE;
  return e == hipSuccess ? FP8BS_OK : FP8BS_EHIP;
}

constexpr int64_t MAX_DIM = int64_t(1) << 30;

// Kernel attributes (dynamic LDS above the default), once per process and device.
fp8bs_status ensure_attributes() {
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return FP8BS_EHIP;
  if (dev < 0 || dev >= 64) return FP8BS_EHIP;
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev]) {
    if (fp8bs::set_layernorm_attributes() != hipSuccess) return FP8BS_EHIP;
    done[dev] = true;
  }
  return FP8BS_OK;
}

fp8bs_status check_workspace(const void* workspace, int64_t have, int64_t need) {
  if (need == 0) return FP8BS_OK;
  if (!workspace || have < need) return FP8BS_EINVAL;
  return aligned(workspace, 16) ? FP8BS_OK : FP8BS_EALIGN;
}

// Sizes and the arguments that both forms of the layer norm have.
fp8bs_status check_layernorm(const void* x, const void* residual, const void* gamma, const void* beta, float eps,
                             int64_t rows, int64_t d, const void* h, const void* y, const float* mean,
                             const float* rstd) {
  if (rows < 0 || d < 0 || !(eps >= 0) || std::isinf(eps) || (mean == nullptr) != (rstd == nullptr))
    return FP8BS_EINVAL;
  if (rows > MAX_DIM || d > fp8bs::layernorm_max_cols() || d % 16) return FP8BS_ESHAPE;
  if (rows == 0 || d == 0) return FP8BS_OK;
  if (!x || !gamma) return FP8BS_EINVAL;
  for (const void* p : {x, residual, gamma, beta, h, y})
    if (!aligned(p, 16)) return FP8BS_EALIGN;
  return aligned(mean, 4) && aligned(rstd, 4) ? FP8BS_OK : FP8BS_EALIGN;
}

constexpr int64_t MAX_MOE_DIM = 32768;

fp8bs_status check_moe_sizes(int64_t tokens, int64_t top, int64_t experts, int64_t hidden, int64_t inner) {
  if (tokens < 0 || top < 1 || experts < 1 || experts > FP8BS_MAX_GROUPS || hidden < 0 || inner < 0)
    return FP8BS_EINVAL;
  if (top > FP8BS_MAX_MOE_CHOICES || tokens > FP8BS_MAX_MOE_CHOICES || tokens * top > FP8BS_MAX_MOE_CHOICES)
    return FP8BS_ESHAPE;
  if (hidden % 16 || hidden > MAX_MOE_DIM || inner % 16 || inner < 16 || inner > MAX_MOE_DIM) return FP8BS_ESHAPE;
  return FP8BS_OK;
}

constexpr int64_t MAX_COUNT = int64_t(1) << 36;  // a launch's chunks of 32 KB stay below 2^31

fp8bs_status check_grads(const void* const* grads, void* const* outs, bool clips, const int64_t* counts,
                         const int32_t* types, int32_t n) {
  if (n < 0 || n > FP8BS_MAX_TENSORS) return FP8BS_EINVAL;
  if (n > 0 && (!grads || !counts || !types || (clips && !outs))) return FP8BS_EINVAL;
  for (int32_t i = 0; i < n; ++i) {
    if (counts[i] < 0 || (types[i] != FP8BS_F32 && types[i] != FP8BS_BF16)) return FP8BS_EINVAL;
    if (counts[i] > MAX_COUNT) return FP8BS_ESHAPE;
    if (counts[i] == 0) continue;
    if (!grads[i] || (clips && !outs[i])) return FP8BS_EINVAL;
    const uintptr_t size = types[i] == FP8BS_F32 ? 4 : 2;
    if (!aligned(grads[i], size) || (clips && !aligned(outs[i], size))) return FP8BS_EALIGN;
  }
  return FP8BS_OK;
}

// Does a tensor that is written overlap another one?  (outs[i] == grads[i] is one tensor.)  The
// norm is one more, read or written while tensors are.
bool overlapping(const void* const* grads, void* const* outs, const int64_t* counts, const int32_t* types,
                 int32_t n, const float* norm, bool norm_written) {
  struct Span {
    uintptr_t begin, end;
    bool written;
  };
  std::vector<Span> spans;
  spans.reserve(2 * (size_t)n + 1);
  spans.push_back({reinterpret_cast<uintptr_t>(norm), reinterpret_cast<uintptr_t>(norm) + 4, norm_written});
  for (int32_t i = 0; i < n; ++i) {
    if (counts[i] == 0) continue;
    const uintptr_t bytes = (uintptr_t)counts[i] * (types[i] == FP8BS_F32 ? 4 : 2);
    const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]), o = reinterpret_cast<uintptr_t>(outs[i]);
    spans.push_back({o, o + bytes, true});
    if (g != o) spans.push_back({g, g + bytes, false});
  }
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t any = 0, written = 0;  // the furthest ends so far
  for (const Span& s : spans) {
    if (s.begin < written || (s.written && s.begin < any)) return true;
    any = std::max(any, s.end);
    if (s.written) written = std::max(written, s.end);
  }
  return false;
}

fp8bs_status check_clip(const void* const* grads, void* const* outs, const int64_t* counts, const int32_t* types,
                        int32_t n, double max_norm, double eps, const float* norm, bool norm_written) {
  const fp8bs_status st = check_grads(grads, outs, true, counts, types, n);
  if (st != FP8BS_OK) return st;
  if (!(max_norm >= 0) || !(eps >= 0) || std::isinf(max_norm) || std::isinf(eps) || !norm) return FP8BS_EINVAL;
  if (!aligned(norm, 4)) return FP8BS_EALIGN;
  try {
    if (overlapping(grads, outs, counts, types, n, norm, norm_written)) return FP8BS_EINVAL;
  } catch (...) {  // no host memory
    return FP8BS_EHIP;
  }
  return FP8BS_OK;
}

}  // namespace

extern "C" {

fp8bs_status fp8bs_layernorm_quantize_tg128(const void* x_bf16, const void* residual_bf16, const void* gamma_bf16,
                                            const void* beta_bf16, float eps, int64_t rows, int64_t d, void* h_bf16,
                                            void* q_e4m3, float* scales, void* y_bf16, float* mean, float* rstd,
                                            void* stream) {
  const fp8bs_status st =
      check_layernorm(x_bf16, residual_bf16, gamma_bf16, beta_bf16, eps, rows, d, h_bf16, y_bf16, mean, rstd);
  if (st != FP8BS_OK || rows == 0 || d == 0) return st;
  if (!q_e4m3 || !scales) return FP8BS_EINVAL;
  if (!aligned(q_e4m3, 16) || !aligned(scales, 4)) return FP8BS_EALIGN;
  return from_launch(fp8bs::launch_layernorm(x_bf16, residual_bf16, gamma_bf16, beta_bf16, eps, rows, d, h_bf16,
                                             q_e4m3, scales, y_bf16, mean, rstd, (hipStream_t)stream));
}

fp8bs_status fp8bs_layernorm(const void* x_bf16, const void* residual_bf16, const void* gamma_bf16,
                             const void* beta_bf16, float eps, int64_t rows, int64_t d, void* h_bf16, void* y_bf16,
                             float* mean, float* rstd, void* stream) {
  const fp8bs_status st =
      check_layernorm(x_bf16, residual_bf16, gamma_bf16, beta_bf16, eps, rows, d, h_bf16, y_bf16, mean, rstd);
  if (st != FP8BS_OK || rows == 0 || d == 0) return st;
  if (!y_bf16) return FP8BS_EINVAL;
  return from_launch(fp8bs::launch_layernorm(x_bf16, residual_bf16, gamma_bf16, beta_bf16, eps, rows, d, h_bf16,
                                             nullptr, nullptr, y_bf16, mean, rstd, (hipStream_t)stream));
}

int64_t fp8bs_layernorm_backward_workspace(int64_t rows, int64_t d) {
  if (rows <= 0 || d <= 0 || rows > MAX_DIM || d > fp8bs::layernorm_max_cols()) return 0;
  return fp8bs::layernorm_backward_workspace(rows, d);
}

fp8bs_status fp8bs_layernorm_backward(const void* dy_bf16, const void* h_bf16, const void* gamma_bf16,
                                      const float* mean, const float* rstd, const void* dresidual_bf16, int64_t rows,
                                      int64_t d, void* dx_bf16, float* dgamma, float* dbeta, int32_t accumulate,
                                      void* workspace, int64_t workspace_bytes, void* stream) {
  if (rows < 0 || d < 0) return FP8BS_EINVAL;
  if (rows > MAX_DIM || d > fp8bs::layernorm_max_cols() || d % 16) return FP8BS_ESHAPE;
  if (d == 0) return FP8BS_OK;
  if (rows > 0 && (!dy_bf16 || !h_bf16 || !gamma_bf16 || !mean || !rstd || !dx_bf16)) return FP8BS_EINVAL;
  for (const void* p : {dy_bf16, h_bf16, gamma_bf16, dresidual_bf16, (const void*)dx_bf16})
    if (!aligned(p, 16)) return FP8BS_EALIGN;
  for (const void* p : {mean, rstd, (const float*)dgamma, (const float*)dbeta})
    if (!aligned(p, 4)) return FP8BS_EALIGN;
  fp8bs_status st = check_workspace(workspace, workspace_bytes, fp8bs_layernorm_backward_workspace(rows, d));
  if (st != FP8BS_OK) return st;
  st = ensure_attributes();
  if (st != FP8BS_OK) return st;
  return from_launch(fp8bs::launch_layernorm_backward(dy_bf16, h_bf16, gamma_bf16, mean, rstd, dresidual_bf16, rows,
                                                      d, dx_bf16, dgamma, dbeta, accumulate != 0, (float*)workspace,
                                                      (hipStream_t)stream));
}

int64_t fp8bs_epilogue_backward_workspace(int64_t rows, int64_t n) {
  if (rows <= 0 || n <= 0 || rows > MAX_DIM || n > MAX_DIM) return 0;
  return fp8bs::epilogue_backward_workspace(rows, n);
}

fp8bs_status fp8bs_epilogue_backward_quantize_tg128(const void* dout_bf16, const void* pre_bf16, int32_t activation,
                                                    int64_t rows, int64_t n, void* dz_bf16, void* q_e4m3,
                                                    float* scales, float* dbias, int32_t accumulate, void* workspace,
                                                    int64_t workspace_bytes, void* stream) {
  if (rows < 0 || n < 0 || activation < FP8BS_ACT_NONE || activation > FP8BS_ACT_SILU) return FP8BS_EINVAL;
  if (rows > MAX_DIM || n > MAX_DIM || n % 16) return FP8BS_ESHAPE;
  if (n == 0) return FP8BS_OK;
  if (rows > 0 && (!dout_bf16 || (!pre_bf16 && activation != FP8BS_ACT_NONE) || !q_e4m3 || !scales))
    return FP8BS_EINVAL;
  for (const void* p : {dout_bf16, pre_bf16, (const void*)dz_bf16, (const void*)q_e4m3})
    if (!aligned(p, 16)) return FP8BS_EALIGN;
  if (!aligned(scales, 4) || !aligned(dbias, 4)) return FP8BS_EALIGN;
  const fp8bs_status st =
      check_workspace(workspace, workspace_bytes, dbias ? fp8bs_epilogue_backward_workspace(rows, n) : 0);
  if (st != FP8BS_OK) return st;
  return from_launch(fp8bs::launch_epilogue_backward(dout_bf16, pre_bf16, activation, rows, n, dz_bf16, q_e4m3,
                                                     scales, dbias, accumulate != 0, (float*)workspace,
                                                     (hipStream_t)stream));
}

int64_t fp8bs_moe_decode_b128_workspace(int64_t tokens, int64_t top, int64_t experts, int64_t hidden,
                                        int64_t inner) {
  if (check_moe_sizes(tokens, top, experts, hidden, inner) != FP8BS_OK || tokens == 0) return 0;
  return fp8bs::moe_decode_workspace((int)tokens, (int)top, (int)experts, hidden, inner);
}

fp8bs_status fp8bs_moe_decode_b128(const void* x_bf16, const int32_t* ids_dev, const float* weights, const void* w1,
                                   const float* s1, const void* w2, const float* s2, const void* residual_bf16,
                                   void* out_bf16, int64_t tokens, int64_t top, int64_t experts, int64_t hidden,
                                   int64_t inner, void* workspace, int64_t workspace_bytes, void* stream) {
  fp8bs_status st = check_moe_sizes(tokens, top, experts, hidden, inner);
  if (st != FP8BS_OK || tokens == 0 || hidden == 0) return st;
  if (!x_bf16 || !ids_dev || !weights || !w1 || !s1 || !w2 || !s2 || !out_bf16) return FP8BS_EINVAL;
  for (const void* p : {x_bf16, w1, w2, residual_bf16, (const void*)out_bf16})
    if (!aligned(p, 16)) return FP8BS_EALIGN;
  for (const void* p : {(const void*)ids_dev, (const void*)weights, (const void*)s1, (const void*)s2})
    if (!aligned(p, 4)) return FP8BS_EALIGN;
  st = check_workspace(workspace, workspace_bytes,
                       fp8bs_moe_decode_b128_workspace(tokens, top, experts, hidden, inner));
  if (st != FP8BS_OK) return st;
  return from_launch(fp8bs::launch_moe_decode(x_bf16, ids_dev, weights, w1, s1, w2, s2, residual_bf16, out_bf16,
                                              (int)tokens, (int)top, (int)experts, hidden, inner, workspace,
                                              (hipStream_t)stream));
}

int64_t fp8bs_grad_norm_workspace(int32_t n) {
  return n < 0 || n > FP8BS_MAX_TENSORS ? 0 : fp8bs::grad_norm_workspace(n);
}

fp8bs_status fp8bs_grad_norm(const void* const* grads, const int64_t* counts, const int32_t* types, int32_t n,
                             float* norm, void* workspace, int64_t workspace_bytes, void* stream) {
  fp8bs_status st = check_grads(grads, nullptr, false, counts, types, n);
  if (st == FP8BS_OK && !norm) st = FP8BS_EINVAL;
  if (st == FP8BS_OK && !aligned(norm, 4)) st = FP8BS_EALIGN;
  if (st == FP8BS_OK) st = check_workspace(workspace, workspace_bytes, fp8bs_grad_norm_workspace(n));
  if (st != FP8BS_OK) return st;
  return from_launch(fp8bs::launch_grad_norm({grads, nullptr, counts, types, n}, norm, (double*)workspace,
                                             (hipStream_t)stream));
}

fp8bs_status fp8bs_clip_grads(const void* const* grads, void* const* outs, const int64_t* counts,
                              const int32_t* types, int32_t n, const float* norm, double max_norm, double eps,
                              void* stream) {
  const fp8bs_status st = check_clip(grads, outs, counts, types, n, max_norm, eps, norm, false);
  if (st != FP8BS_OK) return st;
  return from_launch(fp8bs::launch_clip_grads({grads, outs, counts, types, n}, max_norm, eps,
                                              const_cast<float*>(norm), nullptr, (hipStream_t)stream));
}

fp8bs_status fp8bs_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* counts,
                                  const int32_t* types, int32_t n, double max_norm, double eps, float* norm,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
  fp8bs_status st = check_clip(grads, outs, counts, types, n, max_norm, eps, norm, true);
  if (st == FP8BS_OK) st = check_workspace(workspace, workspace_bytes, fp8bs_grad_norm_workspace(n));
  if (st != FP8BS_OK) return st;
  return from_launch(fp8bs::launch_clip_grads({grads, outs, counts, types, n}, max_norm, eps, norm,
                                              (double*)workspace, (hipStream_t)stream));
}

}  // extern "C"
