// Element-wise part of the gated feed-forward block's backward, for gfx950:
//   dG = dH P1,  dU = dH P2
// with the multipliers the forward kept (gated.hpp).  Rounded to bf16, as which
// they enter the matrix products that follow.  Reads 6 and writes 4 bytes per
// value; bound by memory: 2048 x 11008 in 34 us, 6.6 TB/s (part of it from and to
// the caches).  Formed inside the product with B^T instead, they would not have to
// be read again, but that took longer (68 against 34 + 37 us).
#include "gated.hpp"
#include "kernels.hpp"
#include "timing.hpp"

namespace qlora {

__global__ __launch_bounds__(256) void gated_slopes_kernel(const uint16_t* __restrict__ dH,
                                                           const uint16_t* __restrict__ saved,
                                                           uint16_t* __restrict__ dG, uint16_t* __restrict__ dU,
                                                           int64_t n) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;  // n is a multiple of 8
  if (i >= n) return;
  const u32x4 d = *reinterpret_cast<const u32x4*>(dH + i);
  const u32x4 p1 = *reinterpret_cast<const u32x4*>(saved + i);
  const u32x4 p2 = *reinterpret_cast<const u32x4*>(saved + n + i);
  u32x4 g, u;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float a = bf16_lo(d[q]), b = bf16_hi(d[q]);
    g[q] = pack_bf16x2(a * multiplier(p1[q]), b * multiplier(p1[q] >> 16));
    u[q] = pack_bf16x2(a * multiplier(p2[q]), b * multiplier(p2[q] >> 16));
  }
  *reinterpret_cast<u32x4*>(dG + i) = g;
  *reinterpret_cast<u32x4*>(dU + i) = u;
}

hipError_t launch_gated_slopes(const uint16_t* dH, const uint16_t* saved, uint16_t* dG, uint16_t* dU, int64_t n,
                               hipStream_t s) {
  KernelTimer kt_("gated_slopes_kernel", s);
  hipLaunchKernelGGL(gated_slopes_kernel, dim3((unsigned)((n + 2047) / 2048)), dim3(256), 0, s, dH, saved, dG, dU, n);
  return hipGetLastError();
}

}  // namespace qlora
