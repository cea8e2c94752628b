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
// 4 bytes per element of q and k and one table row per token (4096 tokens of
// 104 heads of 128: 220 MB in 43 us, 5.1 TB/s; 4 tokens of 64 heads 3.5 us, a
// launch).  16 elements to a thread, with 64 bytes of the table from the caches.
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

// A thread turns one unit of one head of a token: 16 elements, 8 pairs of them
// or 16 dims that pass.
template <bool INTER>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
  const uint32_t units = (uint32_t)a.dim / 16;
  const uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t tok = (int64_t)(id / (units * (uint32_t)a.heads));
  if (tok >= a.T) return;
  const uint32_t in_tok = (uint32_t)(id - (uint64_t)tok * (units * (uint32_t)a.heads));
  const int h = (int)(in_tok / units);
  const uint32_t u = in_tok - (uint32_t)h * units;
  int32_t pos = a.t.positions[tok];
  if (pos < 0 || pos >= a.t.n) {
    if (in_tok == 0) atomicOr(a.status, kStatusIndex);
    pos = 0;
  }
  const bool turn = u < (uint32_t)a.t.rot / 16;
  const uint32_t lo = turn && !INTER ? u * 8 : u * 16, hi = turn && !INTER ? lo + (uint32_t)a.t.rot / 2 : lo + 8;
  const bool is_q = h < a.q_heads;
  const int64_t hh = is_q ? h : h - a.q_heads;
  const HeadsView& from = is_q ? a.q : a.k;
  const uint16_t* p = from.data + tok * from.token_stride + hh * from.head_stride;
  u32x4 x = *reinterpret_cast<const u32x4*>(p + lo), y = *reinterpret_cast<const u32x4*>(p + hi);
  if (turn) {
    float cs[16];
    rope_row8(a.t, pos, u * 8, a.sign, cs);
    if (INTER) rope_inter16(x, y, cs);
    else rope_half8(x, y, cs);
  }
  const HeadsView& to = is_q ? a.q_out : a.k_out;
  uint16_t* o = to.data + tok * to.token_stride + hh * to.head_stride;
  *reinterpret_cast<u32x4*>(o + lo) = x;
  *reinterpret_cast<u32x4*>(o + hi) = y;
}

}  // namespace

hipError_t launch_rope_table(const RopeTableArgs& a, float* table, hipStream_t s) {
  const int64_t n = rope_table_threads(a.n, a.rot);
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
  const int64_t n = rope_threads(T, a.heads, dim);
  if (n <= 0) return hipSuccess;
  KernelTimer kt_("rope_kernel", s);
  const dim3 grid((unsigned)((n + 255) / 256));
  if (t.interleaved) hipLaunchKernelGGL(rope_kernel<true>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(rope_kernel<false>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace qlora
