// y = silu(gate) * up with the row quantizer of its result, and its gradient.
//
//   sigma = 1 / (1 + exp(-g)),  y = g sigma u
//   dg = dy u sigma (1 + g (1 - sigma)) = dy u (sigma + g sigma (1 - sigma)),
//   du = dy g sigma
// in fp32 from bf16 inputs; the codes are taken from the fp32 values.  With
// e = exp(-|g|) <= 1 the two sigmoids sigma(|g|) = 1 / (1 + e) and sigma(-|g|) =
// e / (1 + e) never overflow and 1 - sigma loses nothing.  The exponent is split
// into a whole number and a rest of at most 1/2, whose exp2 the hardware takes (a
// rest taken from the rounded exponent costs a far gate more bits the farther it
// lies: 46 x 2^-24 at -60); the reciprocal is the hardware's with one Newton step.
// With one ulp for exp2 sigma(-|g|) is within 2.9 ulp for every gate (where its fp32
// value is not subnormal), and y / 448 was within 3.9 x 2^-24 for every bf16 gate
// of [2^-7, 80] and either sign: an error there moves the scale of a whole group
// and the codes next to a border.
//
// Bound by HBM traffic: 5 bytes per value forward, 12 backward (14 with y).
// Mapping as in quantize_g128.hip: 16 lanes hold a group's 128 columns of one
// row, eight each.
#include "launch_g128.hpp"
#include "quant_g128.hpp"

namespace fp8bs {

struct Sigmoid {
  float s, c;  // sigma(g) and 1 - sigma(g) = sigma(-g)
};

__device__ __forceinline__ Sigmoid sigmoid(float g) {
  constexpr float L_HI = 1.44269502162933349609375f;   // log2(e) rounded to fp32
  constexpr float L_LO = 1.92596299112661746887e-8f;   // the rest
  constexpr float ROUND = 0x1.8p23f;                   // adding it rounds to a whole number, which the low bits hold
  const float a = fminf(__builtin_fabsf(g), 128.0f);   // exp(-128) is below every fp32 value
  const float t = __builtin_fmaf(a, L_HI, ROUND);
  const float n = t - ROUND;
  // n - a log2(e): the first product and sum lose nothing of a far gate
  const float rest = __builtin_fmaf(-a, L_LO, __builtin_fmaf(-a, L_HI, n));
  // 2^24 e, the factor so that a subnormal e keeps its bits until sigma is rounded
  const int up = 24 + __builtin_bit_cast(int, ROUND) - __builtin_bit_cast(int, t);
  const float e = __builtin_ldexpf(__builtin_amdgcn_exp2f(rest), up);
  const float b = __builtin_fmaf(e, 0x1p-24f, 1.0f);  // in [1, 2]
  const float r = __builtin_amdgcn_rcpf(b);
  const float large = __builtin_fmaf(__builtin_fmaf(-b, r, 1.0f), r, r);
  const float small = e * large * 0x1p-24f;
  return g >= 0.0f ? Sigmoid{large, small} : Sigmoid{small, large};
}

// A region is 4 rows x 512 columns of y; a wave takes 128 columns (a group) of the
// four rows.  (Two or four such loads per lane are slower: 8192 x 2048 forward
// 16.2 us against 18.1, backward 37.4 against 39.5.)  LINES as in put_codes8
// (1500 x 4112 with it 10.1 us, without 8.6).
template <bool LINES>
__global__ void __launch_bounds__(256) swiglu_quant_kernel(const uint16_t* __restrict__ gu, int64_t rows, int64_t d,
                                                           uint8_t* __restrict__ q, float* __restrict__ scales,
                                                           uint16_t* __restrict__ y, uint32_t n_regions) {
  const int lane = threadIdx.x & 63;
  const int piece = lane & 15, rsub = lane >> 4;
  const uint32_t nb = (uint32_t)((d + 127) >> 7), quads = (nb + 3) >> 2;
  for (uint32_t id = blockIdx.x; id < n_regions; id += gridDim.x) {
    const uint32_t reg = region_at<LINES>(id, n_regions);
    const uint32_t rb = reg / quads, cb = (reg - rb * quads) * 4 + (threadIdx.x >> 6);
    const int64_t row = (int64_t)rb * 4 + rsub, col = (int64_t)cb * 128 + piece * 8;
    const bool ok = row < rows && col < d;
    const uint16_t* const p = gu + row * 2 * d + col;
    const uint4 wg = ok ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
    const uint4 wu = ok ? *reinterpret_cast<const uint4*>(p + d) : make_uint4(0, 0, 0, 0);
    float gv[8], uv[8], v[8];
    unpack8(wg, gv);
    unpack8(wu, uv);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = gv[i] * sigmoid(gv[i]).s * uv[i];
    const Scale sc = scale_of(row16_max(amax8(v)));
    // every group of the wave on the reciprocal path (the common case): no branches
    const uint2 codes = __all(sc.r != 0.0f || !ok) ? codes8<true>(v, sc) : codes8<false>(v, sc);
    if (ok) {
      put_codes8<LINES>(q + row * d + col, codes);
      if (y != nullptr) *reinterpret_cast<uint4*>(y + row * d + col) = bf16_round8(v);
      if (piece == 0) scales[row * nb + cb] = sc.s;
    }
  }
}

__device__ __forceinline__ void swiglu_grad(float g, float u, float dy, float& dg, float& du, float& y) {
  const Sigmoid k = sigmoid(g);
  const float silu = g * k.s;
  dg = dy * u * __builtin_fmaf(silu, k.c, k.s);  // dy u is exact
  du = dy * silu;
  y = silu * u;
}

// Groups of 128 columns of [dg | du].  HALVES (d a multiple of 128: a group lies
// in one half): a region of 4 rows x 512 columns of d gives the groups of both
// halves from one load of its inputs.  Otherwise a group may reach over the
// middle: regions run over the 2d columns, and a lane takes the half that its
// eight columns lie in (d % 8 == 0; the second needs no `up`); the inputs are then
// read twice.
template <bool HALVES>
__global__ void __launch_bounds__(256) swiglu_backward_kernel(const uint16_t* __restrict__ gu,
                                                              const uint16_t* __restrict__ dy, int64_t rows,
                                                              int64_t d, uint16_t* __restrict__ dgu,
                                                              uint8_t* __restrict__ q, float* __restrict__ scales,
                                                              uint16_t* __restrict__ y, uint32_t n_regions) {
  const int lane = threadIdx.x & 63;
  const int piece = lane & 15, rsub = lane >> 4;
  const uint32_t nb = (uint32_t)((2 * d + 127) >> 7);
  const uint32_t blocks = HALVES ? (uint32_t)(d >> 7) : nb, quads = (blocks + 3) >> 2;
  for (uint32_t id = blockIdx.x; id < n_regions; id += gridDim.x) {
    const uint32_t reg = region_at<HALVES>(id, n_regions);
    const uint32_t rb = reg / quads, cb = (reg - rb * quads) * 4 + (threadIdx.x >> 6);
    const int64_t row = (int64_t)rb * 4 + rsub, out_col = (int64_t)cb * 128 + piece * 8;
    const bool ok = row < rows && out_col < (HALVES ? d : 2 * d);
    const bool second = !HALVES && out_col >= d;
    const int64_t col = second ? out_col - d : out_col;
    const uint16_t* const p = gu + row * 2 * d + col;
    const uint4 wg = ok ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
    const uint4 wu = ok && !second ? *reinterpret_cast<const uint4*>(p + d) : make_uint4(0, 0, 0, 0);
    const uint4 wd = ok ? *reinterpret_cast<const uint4*>(dy + row * d + col) : make_uint4(0, 0, 0, 0);
    float dg[8], du[8], dv[8], yv[8];
    unpack8(wg, dg);
    unpack8(wu, du);
    unpack8(wd, dv);
#pragma unroll
    for (int i = 0; i < 8; ++i) swiglu_grad(dg[i], du[i], dv[i], dg[i], du[i], yv[i]);
    auto put = [&](const float (&v)[8], int64_t at, uint32_t block) __attribute__((always_inline)) {
      const Scale sc = scale_of(row16_max(amax8(v)));
      const uint2 codes = __all(sc.r != 0.0f || !ok) ? codes8<true>(v, sc) : codes8<false>(v, sc);
      if (ok) {
        *reinterpret_cast<uint4*>(dgu + row * 2 * d + at) = bf16_round8(v);
        put_codes8<HALVES>(q + row * 2 * d + at, codes);
        if (piece == 0) scales[row * nb + block] = sc.s;
      }
    };
    if constexpr (HALVES) {
      put(dg, col, cb);
      put(du, col + d, cb + blocks);
    } else {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = second ? du[i] : dg[i];
      put(v, out_col, cb);
    }
    if (y != nullptr && ok && !second) *reinterpret_cast<uint4*>(y + row * d + col) = bf16_round8(yv);
  }
}

hipError_t launch_swiglu_quantize_tg128(const void* gu, int64_t rows, int64_t d, void* q, float* scales, void* y,
                                        hipStream_t stream) {
  const int64_t n_regions = (rows + 3) / 4 * ((d + 511) / 512);
  if (n_regions > MAX_REGIONS) return hipErrorNotSupported;
  const dim3 grid((unsigned)(n_regions < MAX_GRID ? n_regions : MAX_GRID));
  if (d % 128 == 0)
    hipLaunchKernelGGL(swiglu_quant_kernel<true>, grid, dim3(256), 0, stream, (const uint16_t*)gu, rows, d,
                       (uint8_t*)q, scales, (uint16_t*)y, (uint32_t)n_regions);
  else
    hipLaunchKernelGGL(swiglu_quant_kernel<false>, grid, dim3(256), 0, stream, (const uint16_t*)gu, rows, d,
                       (uint8_t*)q, scales, (uint16_t*)y, (uint32_t)n_regions);
  return hipGetLastError();
}

hipError_t launch_swiglu_backward_quantize_tg128(const void* gu, const void* dy, int64_t rows, int64_t d, void* dgu,
                                                 void* q, float* scales, void* y, hipStream_t stream) {
  const bool halves = d % 128 == 0;
  const int64_t n_regions = (rows + 3) / 4 * (((halves ? d : 2 * d) + 511) / 512);
  if (n_regions > MAX_REGIONS) return hipErrorNotSupported;
  const dim3 grid((unsigned)(n_regions < MAX_GRID ? n_regions : MAX_GRID));
  if (halves)
    hipLaunchKernelGGL((swiglu_backward_kernel<true>), grid, dim3(256), 0, stream, (const uint16_t*)gu,
                       (const uint16_t*)dy, rows, d, (uint16_t*)dgu, (uint8_t*)q, scales, (uint16_t*)y,
                       (uint32_t)n_regions);
  else
    hipLaunchKernelGGL((swiglu_backward_kernel<false>), grid, dim3(256), 0, stream, (const uint16_t*)gu,
                       (const uint16_t*)dy, rows, d, (uint16_t*)dgu, (uint8_t*)q, scales, (uint16_t*)y,
                       (uint32_t)n_regions);
  return hipGetLastError();
}

}  // namespace fp8bs
