// C ABI of the 128-value forms (see include/fp8bs_g128.h) and of their product with an
// epilogue (include/fp8bs_layer.h).
// Host-side argument checks, then one launch on the caller's stream.
#include "fp8bs_g128.h"
#include "fp8bs_layer.h"

#include <hip/hip_runtime.h>

#include <mutex>

#include "launch_g128.hpp"
#include "launch_layer.hpp"

namespace {

constexpr int64_t MAX_DIM = int64_t(1) << 30;
constexpr int64_t MAX_K = int64_t(1) << 22;   // byte offsets inside a tile stay below 2^32
constexpr int64_t MAX_THREADS = 0xFFFFFFFF;   // of one launch

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
int64_t blocks128(int64_t n) { return (n + 127) / 128; }

// hipErrorNotSupported from a launcher: the grid would be too large
fp8bs_status from_launch(hipError_t e) {
  if (e == hipErrorNotSupported) return FP8BS_ESHAPE;
  return e == hipSuccess ? FP8BS_OK : FP8BS_EHIP;
}

// Kernel attributes (dynamic LDS above the default), once per process and device.
fp8bs_status ensure_attributes() {
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return FP8BS_EHIP;
  if (dev < 0 || dev >= 64) return FP8BS_EHIP;
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev]) {
    if (fp8bs::set_gemm_g128_attributes() != hipSuccess) return FP8BS_EHIP;
    if (fp8bs::set_wgrad_attributes() != hipSuccess) return FP8BS_EHIP;
    done[dev] = true;
  }
  return FP8BS_OK;
}

fp8bs_status check_gemm(const void* a, const float* sa, const void* bt, const float* sbt, const void* c, int64_t M,
                        int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return FP8BS_EINVAL;
  if (M > MAX_DIM || N > MAX_DIM || K > MAX_K || N % 16 || K % 16) return FP8BS_ESHAPE;
  if (M == 0 || N == 0) return FP8BS_OK;
  if (!c || (K > 0 && (!a || !sa || !bt || !sbt))) return FP8BS_EINVAL;
  if (!aligned(c, 16)) return FP8BS_EALIGN;
  if (K > 0 && (!aligned(a, 16) || !aligned(bt, 16) || !aligned(sa, 4) || !aligned(sbt, 4))) return FP8BS_EALIGN;
  return FP8BS_OK;
}

}  // namespace

extern "C" {

fp8bs_status fp8bs_quantize_tg128(const void* x_bf16, int64_t rows, int64_t cols, void* q_e4m3, float* scales,
                                  void* stream) {
  if (rows < 0 || cols < 0) return FP8BS_EINVAL;
  if (rows > MAX_DIM || cols > MAX_DIM || cols % 16) return FP8BS_ESHAPE;
  if (rows == 0 || cols == 0) return FP8BS_OK;
  if (!x_bf16 || !q_e4m3 || !scales) return FP8BS_EINVAL;
  if (!aligned(x_bf16, 16) || !aligned(q_e4m3, 16) || !aligned(scales, 4)) return FP8BS_EALIGN;
  return from_launch(fp8bs::launch_quantize_tg128(x_bf16, rows, cols, q_e4m3, scales, (hipStream_t)stream));
}

fp8bs_status fp8bs_quantize_b128(const void* x_bf16, int64_t G, int64_t rows, int64_t cols, void* q_e4m3,
                                 float* scales, void* qt_e4m3, float* scales_t, void* stream) {
  if (G < 1 || rows < 0 || cols < 0) return FP8BS_EINVAL;
  if ((qt_e4m3 == nullptr) != (scales_t == nullptr)) return FP8BS_EINVAL;
  if (G > MAX_DIM || rows > MAX_DIM || cols > MAX_DIM || cols % 16) return FP8BS_ESHAPE;
  if (qt_e4m3 && rows % 16) return FP8BS_ESHAPE;
  if (rows == 0 || cols == 0) return FP8BS_OK;
  const int64_t bands = G * blocks128(rows);  // below 2^54
  if (bands > MAX_DIM || bands * blocks128(cols) > MAX_THREADS / 256) return FP8BS_ESHAPE;
  if (!x_bf16 || !q_e4m3 || !scales) return FP8BS_EINVAL;
  if (!aligned(x_bf16, 16) || !aligned(q_e4m3, 16) || !aligned(scales, 4) || !aligned(qt_e4m3, 16) ||
      !aligned(scales_t, 4))
    return FP8BS_EALIGN;
  return from_launch(fp8bs::launch_quantize_b128(x_bf16, G, rows, cols, q_e4m3, scales, qt_e4m3, scales_t,
                                                 (hipStream_t)stream));
}

fp8bs_status fp8bs_gemm_tg128_nt(const void* a, const float* sa, const void* bt, const float* sbt, void* c_bf16,
                                 int64_t M, int64_t N, int64_t K, void* stream) {
  fp8bs_status st = check_gemm(a, sa, bt, sbt, c_bf16, M, N, K);
  if (st != FP8BS_OK || M == 0 || N == 0) return st;
  st = ensure_attributes();
  if (st != FP8BS_OK) return st;
  return from_launch(fp8bs::launch_gemm_g128(a, sa, bt, sbt, nullptr, 1, c_bf16, M, N, K, (hipStream_t)stream));
}

fp8bs_status fp8bs_gemm_tg128_nt_epilogue(const void* a, const float* sa, const void* bt, const float* sbt,
                                          const void* bias_bf16, int32_t activation, const void* residual_bf16,
                                          void* c_bf16, void* pre_bf16, int64_t M, int64_t N, int64_t K,
                                          void* stream) {
  if (activation < FP8BS_ACT_NONE || activation > FP8BS_ACT_SILU) return FP8BS_EINVAL;
  fp8bs_status st = check_gemm(a, sa, bt, sbt, c_bf16, M, N, K);
  if (st != FP8BS_OK || M == 0 || N == 0) return st;
  if (!aligned(bias_bf16, 16) || !aligned(residual_bf16, 16) || !aligned(pre_bf16, 16)) return FP8BS_EALIGN;
  if (pre_bf16 != nullptr && (pre_bf16 == c_bf16 || pre_bf16 == residual_bf16)) return FP8BS_EINVAL;
  st = ensure_attributes();
  if (st != FP8BS_OK) return st;
  const fp8bs::Epilogue e = {(const uint16_t*)bias_bf16, (const uint16_t*)residual_bf16, (uint16_t*)pre_bf16,
                             activation};
  return from_launch(fp8bs::launch_gemm_g128_epilogue(a, sa, bt, sbt, e, c_bf16, M, N, K, (hipStream_t)stream));
}

fp8bs_status fp8bs_grouped_gemm_tg128_nt(const void* a, const float* sa, const void* bt, const float* sbt,
                                         const int32_t* offsets_dev, int32_t G, void* c_bf16, int64_t M_total,
                                         int64_t N, int64_t K, void* stream) {
  if (G < 1 || G > FP8BS_MAX_GROUPS) return FP8BS_EINVAL;
  if (!offsets_dev) return FP8BS_EINVAL;
  if (!aligned(offsets_dev, 4)) return FP8BS_EALIGN;
  fp8bs_status st = check_gemm(a, sa, bt, sbt, c_bf16, M_total, N, K);
  if (st != FP8BS_OK || M_total == 0 || N == 0) return st;
  st = ensure_attributes();
  if (st != FP8BS_OK) return st;
  return from_launch(fp8bs::launch_gemm_g128(a, sa, bt, sbt, offsets_dev, G, c_bf16, M_total, N, K,
                                             (hipStream_t)stream));
}

fp8bs_status fp8bs_grouped_wgrad(const void* dy_bf16, const void* x_bf16, const int32_t* offsets_dev, int32_t G,
                                 float* dw, int32_t accumulate, int64_t M_total, int64_t N, int64_t K, void* stream) {
  if (G < 1 || G > FP8BS_MAX_GROUPS) return FP8BS_EINVAL;
  if (M_total < 0 || N < 0 || K < 0) return FP8BS_EINVAL;
  if (M_total > MAX_DIM || N > MAX_K || K > MAX_K || N % 16 || K % 16) return FP8BS_ESHAPE;
  if (!offsets_dev) return FP8BS_EINVAL;
  if (!aligned(offsets_dev, 4)) return FP8BS_EALIGN;
  if (N == 0 || K == 0) return FP8BS_OK;
  if (!dw || (M_total > 0 && (!dy_bf16 || !x_bf16))) return FP8BS_EINVAL;
  if (!aligned(dw, 16) || !aligned(dy_bf16, 16) || !aligned(x_bf16, 16)) return FP8BS_EALIGN;
  fp8bs_status st = ensure_attributes();
  if (st != FP8BS_OK) return st;
  return from_launch(fp8bs::launch_grouped_wgrad(dy_bf16, x_bf16, offsets_dev, G, dw, accumulate != 0, M_total, N, K,
                                                 (hipStream_t)stream));
}

fp8bs_status fp8bs_swiglu_quantize_tg128(const void* gu_bf16, int64_t rows, int64_t d, void* q_e4m3, float* scales,
                                         void* y_bf16, void* stream) {
  if (rows < 0 || d < 0) return FP8BS_EINVAL;
  if (rows > MAX_DIM || d > MAX_DIM / 2 || d % 16) return FP8BS_ESHAPE;
  if (rows == 0 || d == 0) return FP8BS_OK;
  if (!gu_bf16 || !q_e4m3 || !scales) return FP8BS_EINVAL;
  if (!aligned(gu_bf16, 16) || !aligned(q_e4m3, 16) || !aligned(scales, 4) || !aligned(y_bf16, 16))
    return FP8BS_EALIGN;
  return from_launch(fp8bs::launch_swiglu_quantize_tg128(gu_bf16, rows, d, q_e4m3, scales, y_bf16,
                                                         (hipStream_t)stream));
}

fp8bs_status fp8bs_swiglu_backward_quantize_tg128(const void* gu_bf16, const void* dy_bf16, int64_t rows, int64_t d,
                                                  void* dgu_bf16, void* q_e4m3, float* scales, void* y_bf16,
                                                  void* stream) {
  if (rows < 0 || d < 0) return FP8BS_EINVAL;
  if (rows > MAX_DIM || d > MAX_DIM / 2 || d % 16) return FP8BS_ESHAPE;
  if (rows == 0 || d == 0) return FP8BS_OK;
  if (!gu_bf16 || !dy_bf16 || !dgu_bf16 || !q_e4m3 || !scales) return FP8BS_EINVAL;
  if (!aligned(gu_bf16, 16) || !aligned(dy_bf16, 16) || !aligned(dgu_bf16, 16) || !aligned(q_e4m3, 16) ||
      !aligned(scales, 4) || !aligned(y_bf16, 16))
    return FP8BS_EALIGN;
  return from_launch(fp8bs::launch_swiglu_backward_quantize_tg128(gu_bf16, dy_bf16, rows, d, dgu_bf16, q_e4m3,
                                                                  scales, y_bf16, (hipStream_t)stream));
}

}  // extern "C"
