// Rotary position embedding for gfx950: pair i of a head, (a, b), is turned
// by the angle of its position,
//     a' = a c - b s,   b' = b c + a s,   (c, s) = table[position][i],
// with b half a rotation away (half layout) or next to a (interleaved); dims
// from `rot` on pass through.  The rotation is orthogonal up to the table's
// amplitude, so its gradient is the same kernel with s negated.
//
// The table is built once per model (fp64 angles, rounded to fp32 once), so
// that long positions lose nothing: an fp32 product position * frequency is
// off by position * 2^-24 radians.  The rotation itself is bound by memory:
// 4 bytes per element of q and k and one table row per token.
#include <cmath>

#include "common.hpp"
#include "device_state.hpp"
#include "kvcache.hpp"
#include "rope.hpp"
#include "timing.hpp"

namespace qlora {

namespace {

__global__ __launch_bounds__(256) void rope_table_kernel(RopeTableArgs a, float2* __restrict__ table) {
  const int half = a.rot / 2;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= a.n * half) return;
  const int64_t pos = e / half;
  const int i = (int)(e - pos * half);
  const double two_pi = 6.283185307179586476925286766559;
  double base = a.base;
  if (a.scaling == 2) base *= pow(a.factor, (double)a.rot / (double)(a.rot > 2 ? a.rot - 2 : 1));
  double freq = pow(base, -2.0 * (double)i / (double)a.rot);
  if (a.scaling == 1) freq /= a.factor;
  if (a.scaling == 3) {
    // Turns that this pair makes over the original context: at `high` and
    // more the frequency stays, at `low` and fewer it is divided.
    double keep = (a.original * freq / two_pi - a.low) / (a.high - a.low);
    keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
    freq = freq * keep + freq / a.factor * (1.0 - keep);
  }
  double s, c;
  sincos((double)pos * freq, &s, &c);
  table[e] = make_float2((float)(c * a.amplitude), (float)(s * a.amplitude));
}

struct RopeArgs {
  int64_t T;
  int32_t dim, q_heads, heads;  // heads: q and k together
  RopeTable t;
  float sign;
  HeadsView q, q_out, k, k_out;
  int* status;
};

// A thread turns one unit (16 elements of the dims: 8 pairs, or 16 dims that
// pass) of HB heads of one token, with the unit's table values read once.
template <int HB, bool INTER>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
  const uint32_t units = (uint32_t)a.dim / 16, groups = ((uint32_t)a.heads + HB - 1) / HB;
  const uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  const uint64_t t64 = id / (units * groups);
  if (t64 >= (uint64_t)a.T) return;
  const int64_t tok = (int64_t)t64;
  const uint32_t in_tok = (uint32_t)(id - t64 * (units * groups));
  const uint32_t grp = in_tok / units, u = in_tok - grp * units;
  const uint32_t turned = (uint32_t)a.t.rot / 16;
  int32_t pos = a.t.positions[tok];
  if (pos < 0 || pos >= a.t.n) {
    if (in_tok == 0) atomicOr(a.status, kStatusIndex);
    pos = 0;
  }
  const bool turn = u < turned;
  const uint32_t lo = !turn ? u * 16 : INTER ? u * 16 : u * 8;
  const uint32_t hi = !turn || INTER ? lo + 8 : lo + (uint32_t)a.t.rot / 2;
  float cs[16];
  if (turn) rope_row8(a.t, pos, u * 8, a.sign, cs);
  u32x4 x[HB], y[HB];
#pragma unroll
  for (int j = 0; j < HB; ++j) {
    const int h = (int)(grp * HB) + j;
    if (h < a.heads) {
      const HeadsView& v = h < a.q_heads ? a.q : a.k;
      const uint16_t* p = v.data + tok * v.token_stride + (int64_t)(h < a.q_heads ? h : h - a.q_heads) * v.head_stride;
      x[j] = *reinterpret_cast<const u32x4*>(p + lo);
      y[j] = *reinterpret_cast<const u32x4*>(p + hi);
    }
  }
#pragma unroll
  for (int j = 0; j < HB; ++j) {
    const int h = (int)(grp * HB) + j;
    if (h < a.heads) {
      if (turn) {
        if (INTER) rope_inter16(x[j], y[j], cs);
        else rope_half8(x[j], y[j], cs);
      }
      const HeadsView& v = h < a.q_heads ? a.q_out : a.k_out;
      uint16_t* p = v.data + tok * v.token_stride + (int64_t)(h < a.q_heads ? h : h - a.q_heads) * v.head_stride;
      *reinterpret_cast<u32x4*>(p + lo) = x[j];
      *reinterpret_cast<u32x4*>(p + hi) = y[j];
    }
  }
}

}  // namespace

hipError_t launch_rope_table(const RopeTableArgs& a, float* table, hipStream_t s) {
  const int64_t n = a.n * (a.rot / 2);
  if (n <= 0) return hipSuccess;
  KernelTimer kt_("rope_table_kernel", s);
  hipLaunchKernelGGL(rope_table_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a,
                     reinterpret_cast<float2*>(table));
  return hipGetLastError();
}

hipError_t launch_rope(int64_t T, int32_t dim, const RopeTable& t, bool inverse, const HeadsView& q,
                       const HeadsView& q_out, const HeadsView& k, const HeadsView& k_out, hipStream_t s) {
  RopeArgs a{};
  hipError_t e = hipSuccess;
  a.status = status_word(&e);
  if (!a.status) return e;
  a.T = T;
  a.dim = dim;
  a.q_heads = q.heads;
  a.heads = q.heads + k.heads;
  a.t = t;
  a.sign = inverse ? -1.0f : 1.0f;
  a.q = q;
  a.q_out = q_out;
  a.k = k;
  a.k_out = k_out;
  const int64_t n = T * a.heads * (dim / 16);
  if (n <= 0) return hipSuccess;
  KernelTimer kt_("rope_kernel", s);
  const dim3 grid((unsigned)((n + 255) / 256));
  if (t.interleaved) hipLaunchKernelGGL((rope_kernel<1, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((rope_kernel<1, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace qlora
