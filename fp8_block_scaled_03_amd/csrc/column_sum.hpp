// The second step of sums over rows: partial sums [parts, n], one row for each workgroup
// of the kernel before, are added in order.  Column c goes to first[c] if c < split, else
// to second[c - split]; either may be null (not wanted).  accumulate: added to what
// is there.
//
// A workgroup takes 64 columns; its 16 waves share the parts (wave k takes every
// 16th from k) and are joined in order through LDS.  The partial sums were written
// right before and are read from the caches.
#pragma once
#include "common.hpp"

namespace fp8bs {

static __global__ void __launch_bounds__(1024) column_sum_kernel(const float* __restrict__ partial, int parts,
                                                                 int64_t n, int64_t split,
                                                                 float* __restrict__ first,
                                                                 float* __restrict__ second, bool accumulate) {
  constexpr int AHEAD = 8;  // loads in flight, without conditions (255 parts: the last seven one by one 1.5 us more)
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 64 + lane;
  float s = 0.0f;
  if (c < n) {
    const float* const p = partial + c;
    for (int k0 = w; k0 < parts; k0 += 16 * AHEAD) {
      float v[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) v[i] = p[(k0 + 16 * i < parts ? k0 + 16 * i : k0) * n];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) s += k0 + 16 * i < parts ? v[i] : 0.0f;
    }
  }
  sums[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < n) {
#pragma unroll
    for (int k = 1; k < 16; ++k) s += sums[k][lane];
    float* const out = c < split ? (first ? first + c : nullptr) : (second ? second + (c - split) : nullptr);
    if (out) *out = accumulate ? *out + s : s;
  }
}

static inline void launch_column_sum(const float* partial, unsigned parts, int64_t n, int64_t split, float* first,
                                     float* second, bool accumulate, hipStream_t stream) {
  const int64_t blocks = (n + 63) / 64;
  const unsigned x = (unsigned)(blocks < 65536 ? blocks : 65536);  // (a grid side holds fewer than 2^32 threads)
  hipLaunchKernelGGL(column_sum_kernel, dim3(x, (unsigned)((blocks + x - 1) / x)), dim3(1024), 0, stream, partial,
                     (int)parts, n, split, first, second, accumulate);
}

}  // namespace fp8bs
