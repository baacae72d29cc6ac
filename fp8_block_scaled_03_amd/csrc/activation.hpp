// Activations of a product's epilogue and their derivatives, and the sigmoid that they
// share with the gated activation.
//
//   relu  max(z, 0);   silu  z sigma(z);   gelu_tanh  z sigma(f), f = z (C0 + C1 z^2),
//   C0 = 2 sqrt(2 / pi), C1 = 0.044715 C0  (z (1 + tanh(f / 2)) / 2 is that);
//   gelu  z Phi(z), Phi the normal distribution's function.
//
// With t = |z| and phi(t) = exp(-t^2 / 2) / sqrt(2 pi):
//   Phi(-t) = exp(-t^2 / 2) Q(t),  Q(t) = exp(t^2 / 2) erfc(t / sqrt 2) / 2,
// and Q, which falls from 1/2 to 0.4 / t, is for the gradient 1/2 - v r(v), v = a t / (1 + a t),
// a = 0.28, with a polynomial r of degree 7 (fitted here to the least error on [0, 14.5], which may
// grow as 0.3 t from t = 3 on, as t phi does, beside which Q stands: 0.15 x 2^-24 with the
// coefficients as fp32 holds them).  Near t = 0 the 1/2 is exact, so the roundings of the polynomial and of the
// reciprocal count by the small rest: on normal z of deviation 1.5 the slope is 0.42 x 2^-24 rms off.
// (As u q(u), u = 1 / (1 + a t), with a polynomial of degree 8 all of Q took them: 0.6 to 0.9 x 2^-24.)
//   gelu' = Phi(z) + z phi(z) = S for z < 0 and 1 - S else,
//   S = exp(-t^2 / 2) (Q(t) - t / sqrt(2 pi)).
#pragma once
#include "common.hpp"

namespace fp8bs {

enum Activation { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

constexpr float GT_C0 = 1.5957691669464111f, GT_C0_LO = -4.534068054340423e-08f;  // C0, C1 in two parts
constexpr float GT_C1 = 0.07135481387376785f, GT_C1_LO = 2.3988324659995897e-09f;

struct Sigmoid {
  float s, c;  // sigma(g) and 1 - sigma(g) = sigma(-g)
};

// sigma(g + g_lo), g_lo a correction below g's last bit.  With e = exp(-|g|) <= 1 the two
// sigmoids sigma(|g|) = 1 / (1 + e) and sigma(-|g|) = e / (1 + e) never overflow and
// 1 - sigma loses nothing.  The exponent is split into a whole number and a rest of at
// most 1/2, whose exp2 the hardware takes (a rest taken from the rounded exponent
// costs a far gate more bits the farther it lies: 46 x 2^-24 at -60); the
// reciprocal is the hardware's with one Newton step.  With one ulp for exp2
// sigma(-|g|) is within 2.9 ulp for every gate (where its fp32 value is not subnormal).
template <bool CORRECTED = false>
__device__ __forceinline__ Sigmoid sigmoid(float g, float g_lo = 0.0f) {
  constexpr float L_HI = 1.44269502162933349609375f;   // log2(e) rounded to fp32
  constexpr float L_LO = 1.92596299112661746887e-8f;   // the rest
  constexpr float ROUND = 0x1.8p23f;                   // adding it rounds to a whole number, which the low bits hold
  const float a = fminf(__builtin_fabsf(g), 128.0f);   // exp(-128) is below every fp32 value
  const float t = __builtin_fmaf(a, L_HI, ROUND);
  const float n = t - ROUND;
  // n - a log2(e): the first product and sum lose nothing of a far gate
  float rest = __builtin_fmaf(-a, L_LO, __builtin_fmaf(-a, L_HI, n));
  if constexpr (CORRECTED) rest = __builtin_fmaf(g < 0.0f ? g_lo : -g_lo, L_HI, rest);
  // 2^24 e, the factor so that a subnormal e keeps its bits until sigma is rounded
  const int up = 24 + __builtin_bit_cast(int, ROUND) - __builtin_bit_cast(int, t);
  const float e = __builtin_ldexpf(__builtin_amdgcn_exp2f(rest), up);
  const float b = __builtin_fmaf(e, 0x1p-24f, 1.0f);  // in [1, 2]
  const float r = __builtin_amdgcn_rcpf(b);
  const float large = __builtin_fmaf(__builtin_fmaf(-b, r, 1.0f), r, r);
  const float small = e * large * 0x1p-24f;
  return g >= 0.0f ? Sigmoid{large, small} : Sigmoid{small, large};
}

// Q(t), t >= 0.
__device__ __forceinline__ float normal_tail_ratio(float t) {
  constexpr float A = 0.2800000011920929f;
  const float v = t * A * __builtin_amdgcn_rcpf(__builtin_fmaf(t, A, 1.0f));
  float r = -0.039345093071460724f;
  r = __builtin_fmaf(r, v, 0.09880146384239197f);
  r = __builtin_fmaf(r, v, 0.012369181960821152f);
  r = __builtin_fmaf(r, v, -0.20192770659923553f);
  r = __builtin_fmaf(r, v, -0.13558310270309448f);
  r = __builtin_fmaf(r, v, 1.1047779321670532f);
  r = __builtin_fmaf(r, v, -1.7639546394348145f);
  r = __builtin_fmaf(r, v, 1.424793004989624f);
  return __builtin_fmaf(-v, r, 0.5f);
}

// ---- forward, for results that are rounded to bf16: the exponentials' arguments are
// rounded once (1e-5 of a value at worst with the rest, where the exponential is about to
// vanish; bf16's half step is 3.9e-3), and what lies below 2^-118 may come out as 0.
// z / (1 + exp(-f)).  A far exponential is infinite and its reciprocal 0.
__device__ __forceinline__ float gated(float z, float f) {
  return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(f * -1.44269502162933349609375f));
}
// max(z, 0) - t Phi(-t), with a polynomial of degree 5 in u = 1 / (1 + 0.308 t) for Q(t)
// (4e-6 on [0, 13.3]; beyond, exp(-t^2 / 2) < 2^-127).  t stops at 64, so that no infinity meets a 0.
__device__ __forceinline__ float gelu(float z) {
  const float t = __builtin_elementwise_minimum(__builtin_fabsf(z), 64.0f);
  const float u = __builtin_amdgcn_rcpf(__builtin_fmaf(t, 0.3079999983310699f, 1.0f));
  float q = -0.07553243637084961f;
  q = __builtin_fmaf(q, u, 0.18990986049175262f);
  q = __builtin_fmaf(q, u, 0.006956856697797775f);
  q = __builtin_fmaf(q, u, 0.13669516146183014f);
  q = __builtin_fmaf(q, u, 0.1188424751162529f);
  q = __builtin_fmaf(q, u, 0.12312617152929306f);
  const float tail = __builtin_amdgcn_exp2f(t * t * -0.7213475108146667f) * (q * u);
  return __builtin_fmaf(-t, tail, __builtin_elementwise_maximum(z, 0.0f));
}

// ---- derivatives at a bf16 z, to fp32: the codes of a whole group hang on the
// largest.
template <int ACT>
__device__ __forceinline__ float slope(float z) {
  // far values behave as at these bounds, bit for bit, and overflow nothing; a NaN stays
  auto within = [](float v, float bound) __attribute__((always_inline)) {
    return __builtin_elementwise_minimum(__builtin_elementwise_maximum(v, -bound), bound);
  };
  if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : z != z ? z : 0.0f;
  if constexpr (ACT == ACT_SILU) {
    z = within(z, 256.0f);
    const Sigmoid k = sigmoid(z);
    return __builtin_fmaf(z * k.s, k.c, k.s);
  }
  if constexpr (ACT == ACT_GELU_TANH) {
    // f = z (C0 + C1 z^2) in two parts (z^2 is exact; the product's and the sum's rest, Knuth's
    // two-sum): sigma(f) of a far z needs f's low bits
    z = within(z, 64.0f);
    const float z2 = z * z, m = GT_C1 * z2, m_lo = __builtin_fmaf(GT_C1, z2, -m);
    const float p = m + GT_C0, c = p - m;
    const float p_lo = ((m - (p - c)) + (GT_C0 - c)) + (m_lo + __builtin_fmaf(GT_C1_LO, z2, GT_C0_LO));
    const float f = z * p, f_lo = __builtin_fmaf(z, p_lo, __builtin_fmaf(z, p, -f));
    const Sigmoid k = sigmoid<true>(f, f_lo);
    return __builtin_fmaf(k.s * k.c, z * __builtin_fmaf(3.0f * GT_C1, z2, GT_C0), k.s);
  }
  if constexpr (ACT == ACT_GELU) {
    constexpr float L_HI = 0.7213475108146667f, L_LO = 9.629815167500055e-09f;  // log2(e) / 2
    constexpr float ROUND = 0x1.8p23f;
    const float t = __builtin_elementwise_minimum(__builtin_fabsf(z), 32.0f);
    const float t2 = t * t;                                 // exact: t has eight bits
    const float m = __builtin_fmaf(t2, L_HI, ROUND), n = m - ROUND;
    const float rest = __builtin_fmaf(-t2, L_LO, __builtin_fmaf(-t2, L_HI, n));
    const float e = __builtin_ldexpf(__builtin_amdgcn_exp2f(rest),
                                     __builtin_bit_cast(int, ROUND) - __builtin_bit_cast(int, m));
    const float s = e * __builtin_fmaf(t, -0.3989422917366028f, normal_tail_ratio(t));
    return z < 0.0f ? s : 1.0f - s;
  }
  return 1.0f;
}

}  // namespace fp8bs
