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
// to |g| <= 16, where those have long been reached.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.4426950408889634f));
}
__device__ __forceinline__ void activation(int act, float g, float& a, float& slope) {
  if (act == kActSilu) {
    const float s = sigmoid(g);
    a = g * s;
    slope = s + a * (1.0f - s);
  } else {
    const float c = fminf(fmaxf(g, -16.0f), 16.0f);
    if (act == kActGelu) {  // g Phi(g); erfc keeps the digits of the lower tail
      const float phi = 0.5f * erfcf(-0.70710678118654752f * c);
      a = g * phi;
      slope = phi + c * (0.3989422804014327f * __builtin_amdgcn_exp2f(c * c * -0.72134752044448170f));
    } else {                // 0.5 (1 + tanh y) is the sigmoid of 2 y
      const float c2 = c * c;
      const float s = sigmoid(c * (1.5957691216057308f + 0.07135481282663148f * c2));
      a = g * s;
      slope = s + c * s * (1.0f - s) * (1.5957691216057308f + 0.21406443847989444f * c2);
    }
  }
}

// A multiplier in 16 bits: sign, 6 bits of exponent, 9 of fraction, which is 10
// significant bits from 2^-30 up to 2^33 (below, multiples of 2^-39; from there
// on, infinity).  As bf16 (8 significant bits) the two roundings on the way to a
// gradient would leave it off by 2.9e-3 of the norm; so it is 2.4e-3, its own
// rounding and that of dG and dU as matrix operands.
__device__ __forceinline__ uint32_t multiplier_bits(float x) {
  // 2^-96 moves the exponents that are kept to 0 .. 63; fp32 subnormals become
  // this form's.
  const uint32_t u = __float_as_uint(x * 1.262177448e-29f);
  uint32_t a = u & 0x7FFFFFFFu;
  a = (a + 0x1FFFu + ((a >> 14) & 1u)) >> 14;
  return (a < 0x7FFFu ? a : 0x7FFFu) | (u >> 16 & 0x8000u);
}
__device__ __forceinline__ float multiplier(uint32_t bits) {
  const uint32_t a = bits & 0x7FFFu;
  const float x = a == 0x7FFFu ? INFINITY : __uint_as_float(a << 14) * 7.922816251e28f;
  return __uint_as_float(__float_as_uint(x) | (bits & 0x8000u) << 16);
}

// What a block's output and backward need of one pair of sums.
struct GatedValues {
  float h, p1, p2;
};
__device__ __forceinline__ GatedValues gated_values(int act, float g, float u) {
  float a, slope;
  activation(act, g, a, slope);
  return GatedValues{a * u, slope * u, a};
}

}  // namespace qlora
