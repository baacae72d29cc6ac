// The E4M3 quantizer's steps for groups of 128 columns that 16 neighbouring lanes
// hold (eight values each): the group's maximum and the codes.
#pragma once
#include "common.hpp"
#include "ragged.hpp"

namespace fp8bs {

// Regions of one launch (a workgroup takes every gridDim.x-th).
constexpr int64_t MAX_GRID = 1 << 20, MAX_REGIONS = 0x7FFFFFFF - MAX_GRID;

// Largest value of the 16 lanes of a DPP row, in every one of them (values with
// a clear sign bit, compared as integers).  Lane exchanges inside a row of 16
// go through the VALU: no LDS traffic.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  auto take = [](uint32_t a, uint32_t b) __attribute__((always_inline)) { return a > b ? a : b; };
  v = take(v, __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true));   // lane ^ 1
  v = take(v, __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true));   // lane ^ 2
  v = take(v, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true));  // the other quad of eight
  v = take(v, __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true));  // the other eight
  return v;
}

__device__ __forceinline__ float row16_max(float v) {
  return __builtin_bit_cast(float, row16_max(__builtin_bit_cast(uint32_t, v)));
}

// Largest |x| of eight bf16 values, as fp32 bits.
__device__ __forceinline__ uint32_t amax_bf16x8(uint4 w) {
  typedef unsigned short v2us __attribute__((ext_vector_type(2)));
  auto mag = [](uint32_t x) __attribute__((always_inline)) { return __builtin_bit_cast(v2us, x & 0x7FFF7FFFu); };
  const v2us m = __builtin_elementwise_max(__builtin_elementwise_max(mag(w.x), mag(w.y)),
                                           __builtin_elementwise_max(mag(w.z), mag(w.w)));
  return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
}

struct Scale {
  float s, r;  // scale, and its reciprocal where the reciprocal path is valid (else 0)
};

// amax / 448, rounded to nearest, as in quant_quotient (amax >= QUANT_RECIP_MIN_AMAX).
__device__ __forceinline__ float over_448(float amax) {
  constexpr float R = 1.0f / 448.0f;
  const float q0 = amax * R;
  return __builtin_fmaf(-__builtin_fmaf(q0, 448.0f, -amax), R, q0);
}

__device__ __forceinline__ Scale scale_of(float amax) {
  if (amax >= QUANT_RECIP_MIN_AMAX) {
    const float s = over_448(amax);
    return {s, 1.0f / s};
  }
  return {amax / 448.0f, 0.0f};
}
__device__ __forceinline__ Scale scale_of(uint32_t amax_bits) {
  return scale_of(__builtin_bit_cast(float, amax_bits));
}

// RN32(x / s) from r = RN32(1 / s): q0 = RN(x r), the exact remainder with its sign
// turned (q0 s - x), then RN(q0 - remainder r) (Markstein, IBM J. Res. Dev.
// 34(1), 1990; the same value as quant_quotient_recip).  In this form a zero keeps
// x's sign by itself: for x = -0 the remainder is +0 and -0 - 0 is -0.
__device__ __forceinline__ float quant_quotient(float x, float s, float r) {
  const float q0 = x * r;
  return __builtin_fmaf(-__builtin_fmaf(q0, s, -x), r, q0);
}

// Eight values -> eight codes.  With the reciprocal path |x / s| is at most
// 448 (1 + 2^-22), which rounds to 448, so nothing is clamped; a subnormal scale
// can be off by more, and the division path clamps.
template <bool RECIP>
__device__ __forceinline__ uint2 codes8(const float (&v)[8], Scale k) {
  uint32_t p[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[4 * h + i];
      t[i] = RECIP || k.r != 0.0f ? quant_quotient(x, k.s, k.r) : sat448(quant_quotient_div(x, k.s));
    }
    p[h] = pack_e4m3x4(t[0], t[1], t[2], t[3]);
  }
  return make_uint2(p[0], p[1]);
}

// Largest |v| of eight values.
__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float m = __builtin_fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, __builtin_fabsf(v[i]));
  return m;
}

__device__ __forceinline__ void unpack8(uint4 w, float (&v)[8]) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(ws[i]);
    v[2 * i + 1] = bf16_hi(ws[i]);
  }
}

// fp32 -> bf16, nearest even, two at a time in one instruction.
__device__ __forceinline__ uint32_t bf16_round_pair(float lo, float hi) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{lo, hi}, v2bf));
}
__device__ __forceinline__ uint4 bf16_round8(const float (&v)[8]) {
  return make_uint4(bf16_round_pair(v[0], v[1]), bf16_round_pair(v[2], v[3]), bf16_round_pair(v[4], v[5]),
                    bf16_round_pair(v[6], v[7]));
}

// Eight codes of a lane.  LINES: the rows of codes are multiples of 128, so each line
// has one writer and is written past the caches; else neighbouring regions share
// lines, and their writes meet in the L2 of the XCD that has the run of both.
template <bool LINES>
__device__ __forceinline__ void put_codes8(uint8_t* dst, uint2 codes) {
  if constexpr (LINES) store_codes8(dst, codes.x, codes.y);
  else *reinterpret_cast<uint2*>(dst) = codes;
}
template <bool LINES>
__device__ __forceinline__ uint32_t region_at(uint32_t id, uint32_t n_regions) {
  return LINES ? id : xcd_run(id, n_regions);
}

}  // namespace fp8bs
