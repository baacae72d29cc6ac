// y = silu(gate) * up with the row quantizer of its result, and its gradient.
//
//   sigma = 1 / (1 + exp(-g)),  y = g sigma u
//   dg = dy u sigma (1 + g (1 - sigma)),  du = dy g sigma
// in fp32 from bf16 inputs; the codes are taken from the fp32 values.  With
// e = exp(-|g|) <= 1 the two sigmoids sigma(|g|) = 1 / (1 + e) and sigma(-|g|) =
// e / (1 + e) never overflow and 1 - sigma loses nothing.  e is 2^-t with
// t = |g| log2(e) carried in two parts, so that the hardware's exp2 sees a
// rounded t and the rest enters as a first-order factor; the reciprocal is the
// hardware's with one Newton step.  Both are within about 1.5 ulp, the order
// of the rounding of the products around them: an error there moves the scale
// of a whole group and the codes next to a border.
//
// Bound by HBM traffic: 5 bytes per value forward, 12 backward (14 with y).
// Mapping as in quantize_g128.hip: 16 lanes hold a group's 128 columns of one
// row, eight each.
#include "launch_g128.hpp"
#include "quant_g128.hpp"

#include <type_traits>

namespace fp8bs {

struct Sigmoid {
  float s, c;  // sigma(g) and 1 - sigma(g) = sigma(-g)
};

__device__ __forceinline__ Sigmoid sigmoid(float g) {
  constexpr float L_HI = 1.44269502162933349609375f;   // log2(e) rounded to fp32
  constexpr float L_LO = 1.92596299112661746887e-8f;   // the rest
  const float a = fminf(__builtin_fabsf(g), 128.0f);   // exp(-128) is below every fp32 value
  const float t = a * L_HI;
  const float rest = __builtin_fmaf(a, L_LO, __builtin_fmaf(a, L_HI, -t));
  // the hardware's exp2 flushes subnormal results: far gates are shifted by 2^64
  // (64 - t is exact) and shifted back by the last product
  const bool far = t > 64.0f;
  float e = __builtin_amdgcn_exp2f((far ? 64.0f : 0.0f) - t);
  e = __builtin_fmaf(e * -0.693147180559945f, rest, e);
  const float back = far ? 0x1p-64f : 1.0f;
  const float b = 1.0f + e * back;  // in [1, 2]
  const float r = __builtin_amdgcn_rcpf(b);
  const float large = __builtin_fmaf(__builtin_fmaf(-b, r, 1.0f), r, r);
  const float small = e * large * back;
  return g >= 0.0f ? Sigmoid{large, small} : Sigmoid{small, large};
}

// One wave per region of 4U rows x 128 columns of y.
template <int U>
__global__ void __launch_bounds__(256) swiglu_quant_kernel(const uint16_t* __restrict__ gu, int64_t rows, int64_t d,
                                                           uint8_t* __restrict__ q, float* __restrict__ scales,
                                                           uint16_t* __restrict__ y, int64_t n_regions) {
  const int lane = threadIdx.x & 63;
  const int piece = lane & 15, rsub = lane >> 4;
  const int64_t nb = (d + 127) >> 7;
  const int64_t waves_total = (int64_t)gridDim.x * 4;
  for (int64_t reg = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); reg < n_regions; reg += waves_total) {
    const int64_t rb = reg / nb, cb = reg - rb * nb;
    const int64_t col = cb * 128 + piece * 8;
    uint4 wg[U], wu[U];
    bool ok[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t row = rb * (4 * U) + 4 * k + rsub;
      ok[k] = row < rows && col < d;
      const uint16_t* const p = gu + row * 2 * d + col;
      wg[k] = ok[k] ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
      wu[k] = ok[k] ? *reinterpret_cast<const uint4*>(p + d) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t row = rb * (4 * U) + 4 * k + rsub;
      float gv[8], uv[8], v[8];
      unpack8(wg[k], gv);
      unpack8(wu[k], uv);
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = gv[i] * sigmoid(gv[i]).s * uv[i];
        const uint32_t b = __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu;
        m = m > b ? m : b;
      }
      const Scale sc = scale_of(row16_max(m));
      const uint2 p = __all(sc.r != 0.0f || !ok[k]) ? codes8<true>(v, sc) : codes8<false>(v, sc);
      if (ok[k]) {
        store_codes8(q + row * d + col, p.x, p.y);
        if (y != nullptr) *reinterpret_cast<uint4*>(y + row * d + col) = bf16_round8(v);
        if (piece == 0) scales[row * nb + cb] = sc.s;
      }
    }
  }
}

__device__ __forceinline__ void swiglu_grad(float g, float u, float dy, float& dg, float& du, float& y) {
  const Sigmoid k = sigmoid(g);
  const float silu = g * k.s;
  dg = dy * u * (k.s * (1.0f + g * k.c));
  du = dy * silu;
  y = silu * u;
}

// Groups of 128 columns of [dg | du].  HALVES (d a multiple of 128: a group lies
// in one half): a region of 4U rows x 128 columns of d gives the two groups of
// both halves from one load of its inputs.  Otherwise a group may reach over
// the middle: regions run over the 2d columns, and a lane takes the half that
// its eight columns lie in (d % 8 == 0); the inputs are then read twice, mostly
// from the L2.
template <int U, bool HALVES>
__global__ void __launch_bounds__(256) swiglu_backward_kernel(const uint16_t* __restrict__ gu,
                                                              const uint16_t* __restrict__ dy, int64_t rows,
                                                              int64_t d, uint16_t* __restrict__ dgu,
                                                              uint8_t* __restrict__ q, float* __restrict__ scales,
                                                              uint16_t* __restrict__ y, int64_t n_regions) {
  const int lane = threadIdx.x & 63;
  const int piece = lane & 15, rsub = lane >> 4;
  const int64_t nb = (2 * d + 127) >> 7;
  const int64_t regs_per_row = HALVES ? d >> 7 : nb;
  const int64_t waves_total = (int64_t)gridDim.x * 4;
  for (int64_t reg = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); reg < n_regions; reg += waves_total) {
    const int64_t rb = reg / regs_per_row, cb = reg - rb * regs_per_row;
    const int64_t out_col = cb * 128 + piece * 8;
    const bool second = !HALVES && out_col >= d;
    const int64_t col = second ? out_col - d : out_col;
    uint4 wg[U], wu[U], wd[U];
    bool ok[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t row = rb * (4 * U) + 4 * k + rsub;
      ok[k] = row < rows && out_col < 2 * d;
      const uint16_t* const p = gu + row * 2 * d + col;
      wg[k] = ok[k] ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
      wu[k] = ok[k] ? *reinterpret_cast<const uint4*>(p + d) : make_uint4(0, 0, 0, 0);
      wd[k] = ok[k] ? *reinterpret_cast<const uint4*>(dy + row * d + col) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t row = rb * (4 * U) + 4 * k + rsub;
      float gv[8], uv[8], dv[8], yv[8];
      unpack8(wg[k], gv);
      unpack8(wu[k], uv);
      unpack8(wd[k], dv);
#pragma unroll
      for (int i = 0; i < 8; ++i) swiglu_grad(gv[i], uv[i], dv[i], gv[i], uv[i], yv[i]);  // gv: dg, uv: du
      auto put = [&](const float (&v)[8], int64_t at, int64_t block) __attribute__((always_inline)) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t b = __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu;
          m = m > b ? m : b;
        }
        const Scale sc = scale_of(row16_max(m));
        const uint2 p = __all(sc.r != 0.0f || !ok[k]) ? codes8<true>(v, sc) : codes8<false>(v, sc);
        if (ok[k]) {
          *reinterpret_cast<uint4*>(dgu + row * 2 * d + at) = bf16_round8(v);
          store_codes8(q + row * 2 * d + at, p.x, p.y);
          if (piece == 0) scales[row * nb + block] = sc.s;
        }
      };
      if constexpr (HALVES) {
        put(gv, col, cb);
        put(uv, col + d, cb + (d >> 7));
      } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = second ? uv[i] : gv[i];
        put(v, out_col, cb);
      }
      if (y != nullptr && ok[k] && !second) *reinterpret_cast<uint4*>(y + row * d + col) = bf16_round8(yv);
    }
  }
}

hipError_t launch_swiglu_quantize_tg128(const void* gu, int64_t rows, int64_t d, void* q, float* scales, void* y,
                                        hipStream_t stream) {
  const int64_t nb = (d + 127) / 128;
  auto go = [&](auto U_) {
    constexpr int U = decltype(U_)::value;
    const int64_t n_regions = ((rows + 4 * U - 1) / (4 * U)) * nb;
    int64_t grid = (n_regions + 3) / 4;
    if (grid > 65536) grid = 65536;
    hipLaunchKernelGGL((swiglu_quant_kernel<U>), dim3((unsigned)grid), dim3(256), 0, stream, (const uint16_t*)gu,
                       rows, d, (uint8_t*)q, scales, (uint16_t*)y, n_regions);
  };
  if ((rows + 15) / 16 * nb >= 4096) go(std::integral_constant<int, 4>{});
  else go(std::integral_constant<int, 1>{});
  return hipGetLastError();
}

hipError_t launch_swiglu_backward_quantize_tg128(const void* gu, const void* dy, int64_t rows, int64_t d, void* dgu,
                                                 void* q, float* scales, void* y, hipStream_t stream) {
  auto go = [&](auto U_, auto HALVES_) {
    constexpr int U = decltype(U_)::value;
    constexpr bool HALVES = decltype(HALVES_)::value;
    const int64_t n_regions = ((rows + 4 * U - 1) / (4 * U)) * (HALVES ? d / 128 : (2 * d + 127) / 128);
    int64_t grid = (n_regions + 3) / 4;
    if (grid > 65536) grid = 65536;
    hipLaunchKernelGGL((swiglu_backward_kernel<U, HALVES>), dim3((unsigned)grid), dim3(256), 0, stream,
                       (const uint16_t*)gu, (const uint16_t*)dy, rows, d, (uint16_t*)dgu, (uint8_t*)q, scales,
                       (uint16_t*)y, n_regions);
  };
  const bool many = (rows + 7) / 8 * ((d + 127) / 128) >= 4096;
  if (d % 128 == 0) {
    if (many) go(std::integral_constant<int, 2>{}, std::true_type{});
    else go(std::integral_constant<int, 1>{}, std::true_type{});
  } else {
    if (many) go(std::integral_constant<int, 2>{}, std::false_type{});
    else go(std::integral_constant<int, 1>{}, std::false_type{});
  }
  return hipGetLastError();
}

}  // namespace fp8bs
