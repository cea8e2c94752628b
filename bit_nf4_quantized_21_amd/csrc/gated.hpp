// The gated feed-forward block's activations on the device, and the 16-bit
// form in which its forward keeps what the backward multiplies by.
//
//   H = act(G) U,   dG = dH P1,  dU = dH P2   with  P1 = act'(G) U,  P2 = act(G)
//
// Keeping P1 and P2 instead of G and U leaves the backward no activation to
// compute and one rounding less: both come from the fp32 sums.
#pragma once

#include "common.hpp"

namespace qlora {

constexpr int kActSilu = 0, kActGelu = 1, kActGeluTanh = 2, kActs = 3;

// act(g) and act'(g).  Sigmoids of large arguments reach 0 and 1 through
// exponentials that overflow or vanish; the polynomials beside them are held
// to |g| <= 16, where those have long been reached.  A slope's last term takes g
// itself, not what it is held to (the density is 0 there), so that a g that is no
// number gives a slope that is none.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.4426950408889634f));
}
// Phi(-x) for 0 <= x <= 18 relative to the density's e = exp(-x^2 / 2), which
// keeps the digits of the tail: erfc(z) e^(z^2) / 2 as t times a polynomial in
// t = 1 / (1 + 0.3 z), z = x / sqrt 2.  Its coefficients are a least-squares fit,
// reweighted until the largest relative error (3e-8; with fp32's roundings
// 5e-7) was the same everywhere.
__device__ __forceinline__ float normal_tail(float x, float e) {
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.21213203435596426f * x);
  float q = -0.12786659213149337f;
  q = __builtin_fmaf(q, t, 0.47773531032800365f);
  q = __builtin_fmaf(q, t, -0.49654839726030936f);
  q = __builtin_fmaf(q, t, 0.5302058535986339f);
  q = __builtin_fmaf(q, t, -0.08285859935615333f);
  q = __builtin_fmaf(q, t, 0.21002077108644135f);
  q = __builtin_fmaf(q, t, 0.14956776480930237f);
  q = __builtin_fmaf(q, t, 0.17054613104581406f);
  q = __builtin_fmaf(q, t, 0.16919778363990548f);
  return 0.5f * t * q * e;
}
template <int ACT>
__device__ __forceinline__ void activation(float g, float& a, float& slope) {
  if constexpr (ACT == kActSilu) {
    const float s = sigmoid(g);
    a = g * s;
    slope = s + a * (1.0f - s);
  } else {
    const float c = fminf(fmaxf(g, -16.0f), 16.0f);
    if constexpr (ACT == kActGelu) {  // g Phi(g)
      const float e = __builtin_amdgcn_exp2f(c * c * -0.72134752044448170f);
      const float tail = normal_tail(fabsf(c), e);
      const float phi = c < 0.0f ? tail : 1.0f - tail;
      a = g * phi;
      slope = phi + g * (0.3989422804014327f * e);
    } else {                          // 0.5 (1 + tanh y) is the sigmoid of 2 y
      const float c2 = c * c;
      const float s = sigmoid(c * (1.5957691216057308f + 0.07135481282663148f * c2));
      a = g * s;
      slope = s + g * s * (1.0f - s) * (1.5957691216057308f + 0.21406443847989444f * c2);
    }
  }
}

// A multiplier in 16 bits: sign, 6 bits of exponent, 9 of fraction, which is 10
// significant bits from 2^-30 up to 2^33 (below, multiples of 2^-39; from there
// on, and for what is no number, infinity), rounded to nearest, ties away from zero.  As bf16 (8 significant
// bits) the two roundings on the way to a gradient would leave it off by 2.9e-3
// of the norm; so it is 2.4e-3, its own rounding and that of dG and dU as matrix
// operands.  multiplier_top leaves the 16 bits in the upper half.
__device__ __forceinline__ uint32_t multiplier_top(float x) {
  // 2^-96 moves the exponents that are kept to 0 .. 63 (fp32 subnormals become
  // this form's); what is larger, and NaN, meets the code of infinity.
  const float y = __builtin_amdgcn_fmed3f(x * 1.262177448353619e-29f, -1.0830853e-19f, 1.0830853e-19f);
  const uint32_t u = __float_as_uint(y) + 0x2000u;
  return ((u << 2) & 0x7FFFFFFFu) | (u & 0x80000000u);
}
__device__ __forceinline__ uint32_t multiplier_pair(float lo, float hi) {
  return __builtin_amdgcn_perm(multiplier_top(hi), multiplier_top(lo), 0x07060302u);
}
__device__ __forceinline__ float multiplier(uint32_t bits) {
  const uint32_t a = bits & 0x7FFFu;
  const float x = a == 0x7FFFu ? INFINITY : __uint_as_float(a << 14) * 7.922816251426434e28f;
  return __uint_as_float(__float_as_uint(x) | (bits & 0x8000u) << 16);
}

// What a block's output and backward need of one pair of sums.
struct GatedValues {
  float h, p1, p2;
};
template <int ACT>
__device__ __forceinline__ GatedValues gated_values(float g, float u) {
  float a, slope;
  activation<ACT>(g, a, slope);
  return GatedValues{a * u, slope * u, a};
}
__device__ __forceinline__ GatedValues gated_values(int act, float g, float u) {
  return act == kActSilu ? gated_values<kActSilu>(g, u) : act == kActGelu ? gated_values<kActGelu>(g, u)
                                                                          : gated_values<kActGeluTanh>(g, u);
}

}  // namespace qlora
