// Device arithmetic of the rotation, shared by the rope kernel and the cache
// write.
#pragma once

#include "common.hpp"
#include "kvcache.hpp"

namespace qlora {

// (cos, sin) of the 8 pairs from pair i0 on at a position: cs[2j], cs[2j+1];
// the sines times `sign`.
__device__ __forceinline__ void rope_row8(const RopeTable& t, int64_t pos, uint32_t i0, float sign, float (&cs)[16]) {
  const float4* row = reinterpret_cast<const float4*>(t.table + pos * t.rot + 2 * i0);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 v = row[j];
    cs[4 * j] = v.x;
    cs[4 * j + 1] = v.y * sign;
    cs[4 * j + 2] = v.z;
    cs[4 * j + 3] = v.w * sign;
  }
}

// One pair, each product and sum rounded to fp32 (no contraction, so that the
// same values come out wherever a pair is turned).
__device__ __forceinline__ void rope_pair(float& a, float& b, float c, float s) {
#pragma clang fp contract(off)
  const float ac = a * c, bs = b * s, bc = b * c, as = a * s;
  a = ac - bs;
  b = bc + as;
}

// Half layout: x holds the first elements of 8 pairs, y the second ones.
__device__ __forceinline__ void rope_half8(u32x4& x, u32x4& y, const float (&cs)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float a0 = bf16_lo(x[q]), a1 = bf16_hi(x[q]), b0 = bf16_lo(y[q]), b1 = bf16_hi(y[q]);
    rope_pair(a0, b0, cs[4 * q], cs[4 * q + 1]);
    rope_pair(a1, b1, cs[4 * q + 2], cs[4 * q + 3]);
    x[q] = pack_bf16x2(a0, a1);
    y[q] = pack_bf16x2(b0, b1);
  }
}

// Interleaved layout: dword q of (x, y) is pair q.
__device__ __forceinline__ void rope_inter16(u32x4& x, u32x4& y, const float (&cs)[16]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t w = q < 4 ? x[q & 3] : y[q & 3];
    float a = bf16_lo(w), b = bf16_hi(w);
    rope_pair(a, b, cs[2 * q], cs[2 * q + 1]);
    if (q < 4) x[q & 3] = pack_bf16x2(a, b);
    else y[q & 3] = pack_bf16x2(a, b);
  }
}

}  // namespace qlora
