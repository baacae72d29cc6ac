// Internal launcher declarations of the 128-value forms (include/fp8bs_g128.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bs {
hipError_t launch_quantize_tg128(const void* x, int64_t rows, int64_t cols, void* q, float* scales,
                                 hipStream_t stream);
// qt / scales_t may be null
hipError_t launch_quantize_b128(const void* x, int64_t G, int64_t rows, int64_t cols, void* q, float* scales,
                                void* qt, float* scales_t, hipStream_t stream);
// offsets == null: one range, all M rows (G == 1)
hipError_t launch_gemm_g128(const void* a, const float* sa, const void* bt, const float* sbt, const int32_t* offsets,
                            int G, void* c, int64_t M, int64_t N, int64_t K, hipStream_t stream);
hipError_t set_gemm_g128_attributes();
hipError_t launch_grouped_wgrad(const void* dy, const void* x, const int32_t* offsets, int G, float* dw,
                                bool accumulate, int64_t M_total, int64_t N, int64_t K, hipStream_t stream);
hipError_t set_wgrad_attributes();
hipError_t launch_swiglu_quantize_tg128(const void* gu, int64_t rows, int64_t d, void* q, float* scales, void* y,
                                        hipStream_t stream);
hipError_t launch_swiglu_backward_quantize_tg128(const void* gu, const void* dy, int64_t rows, int64_t d, void* dgu,
                                                 void* q, float* scales, void* y, hipStream_t stream);
}  // namespace fp8bs
