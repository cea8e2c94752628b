// The paged key/value cache: rows are quantized as they are written and
// dequantized as they are read back (gfx950).
//
// A row is one token's `dim` keys (or values) of one head.  With
// top = max |x| over the row and u = fl(1 / top):
//   bf16  x, rounded once;
//   int8  code = rint(x * fl(127 u)), scale = fl(top * fl(1/127));
//   nf4, int4, fp4  y = fl(x u), code of level #{j : y > m_j} over the type's
//         fp32 level boundaries m_j, scale = top;
// all in fp32.  A row with top < 1e-30 is stored as zeros (1/top would leave
// the normal range); a row holding an infinity or a NaN gets a NaN scale, so
// it reads back as NaN instead of as a finite row.  One scale per row (not
// per block of 64) lets attention apply it to whole scores and weights.
//
// Both kernels are bound by memory: 2 bytes per element on the dense side,
// the row's codes and 4 bytes on the other.
#include "common.hpp"
#include "device_state.hpp"
#include "kvcache.hpp"
#include "rope.hpp"
#include "timing.hpp"

namespace qlora {

namespace {

constexpr float kTinyRow = 1e-30f;

struct Decision4 {
  float m[15];
  uint64_t codes;
  uint32_t zero_code;
};

struct KVWriteArgs {
  KVPool pool;
  HeadsView k, v;
  int64_t rows;  // tokens * heads * 2
  const int64_t* slots;
  RopeTable rope;
  Decision4 d4;
  int* status;
};

// 8 elements of a head from element e0, widened, rotated when asked.
template <int ROPE>
__device__ __forceinline__ void load8(const uint16_t* p, uint32_t e0, const RopeTable& t, int64_t pos, bool rotate,
                                      float (&v)[8]) {
  const u32x4 w = *reinterpret_cast<const u32x4*>(p + e0);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    v[2 * q] = bf16_lo(w[q]);
    v[2 * q + 1] = bf16_hi(w[q]);
  }
  if (ROPE == 0 || !rotate || e0 >= (uint32_t)t.rot) return;
  const uint32_t half = (uint32_t)t.rot / 2;
  if (ROPE == 1) {
    const bool first = e0 < half;
    const u32x4 o = *reinterpret_cast<const u32x4*>(p + (first ? e0 + half : e0 - half));
    float cs[16];
    rope_row8(t, pos, first ? e0 : e0 - half, 1.0f, cs);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float other = j & 1 ? bf16_hi(o[j / 2]) : bf16_lo(o[j / 2]);
      if (first) rope_pair(v[j], other, cs[2 * j], cs[2 * j + 1]);
      else rope_pair(other, v[j], cs[2 * j], cs[2 * j + 1]);
    }
  } else {
    const float4* row = reinterpret_cast<const float4*>(t.table + pos * t.rot + e0);
    const float4 r0 = row[0], r1 = row[1];
    rope_pair(v[0], v[1], r0.x, r0.y);
    rope_pair(v[2], v[3], r0.z, r0.w);
    rope_pair(v[4], v[5], r1.x, r1.y);
    rope_pair(v[6], v[7], r1.z, r1.w);
  }
}

// LPR lanes per row, 16 elements per lane.
template <int KT, int LPR, int ROPE>
__global__ __launch_bounds__(256) void kv_write_kernel(KVWriteArgs a) {
  const int64_t r = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  if (r >= a.rows) return;  // the lanes of a row leave together
  const uint32_t H = (uint32_t)a.pool.heads;
  const int64_t ts = r / H;
  const uint32_t h = (uint32_t)(r - ts * H);
  const bool is_v = ts & 1;
  const int64_t tok = ts >> 1;
  const int64_t slot = a.slots[tok];
  if (slot < 0) return;
  const int u = threadIdx.x % LPR;
  if (slot >= (a.pool.pages << a.pool.shift)) {
    if (u == 0) atomicOr(a.status, kStatusIndex);
    return;
  }
  const HeadsView& hv = is_v ? a.v : a.k;
  const uint16_t* p = hv.data + tok * hv.token_stride + (int64_t)h * hv.head_stride;
  int64_t pos = 0;
  if (ROPE && !is_v) {
    pos = a.rope.positions[tok];
    if (pos < 0 || pos >= a.rope.n) {
      if (u == 0) atomicOr(a.status, kStatusIndex);
      pos = 0;
    }
  }
  float v[16] = {};
  const bool mine = u * 16 < a.pool.dim;
  if (mine) {
    float lo[8], hi[8];
    load8<ROPE>(p, u * 16, a.rope, pos, !is_v, lo);
    load8<ROPE>(p, u * 16 + 8, a.rope, pos, !is_v, hi);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = lo[j];
      v[8 + j] = hi[j];
    }
  }
  const int64_t mask = ((int64_t)1 << a.pool.shift) - 1;
  const int64_t row = (((slot >> a.pool.shift) * H + h) << a.pool.shift) + (slot & mask);
  uint8_t* dst = (is_v ? a.pool.v : a.pool.k) + row * kv_row_bytes(a.pool.type, a.pool.dim);
  if (KT == kKVBF16) {
    if (mine) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
        reinterpret_cast<u32x4*>(dst)[2 * u + q] =
            u32x4{pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                  pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7])};
    }
    return;
  }
  // The row's largest magnitude, as integers: NaN > infinity > every number.
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t b = __float_as_uint(v[j]) & 0x7FFFFFFFu;
    top = b > top ? b : top;
  }
#pragma unroll
  for (int off = 1; off < LPR; off <<= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)top, off, 64);
    top = o > top ? o : top;
  }
  const float t = __uint_as_float(top);
  const bool fine = t >= kTinyRow;
  const float unit = fine ? 1.0f / t : 0.0f;
  float* sc = (is_v ? a.pool.vs : a.pool.ks) + row;
  if (u == 0) {
    float s = KT == kKVINT8 ? t * (float)(1.0 / 127.0) : t;
    if (!fine) s = 0.0f;
    if (top >= 0x7F800000u) s = __uint_as_float(0x7FC00000u);
    *sc = s;
  }
  if (!mine) return;
  if (KT == kKVINT8) {
    const float m = unit * 127.0f;
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      w[q] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float c = rintf(v[4 * q + j] * m);
        c = c < -127.0f ? -127.0f : c > 127.0f ? 127.0f : c;
        w[q] |= ((uint32_t)(int)c & 0xFFu) << (8 * j);
      }
    }
    reinterpret_cast<u32x4*>(dst)[u] = u32x4{w[0], w[1], w[2], w[3]};
  } else {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float y = v[j] * unit;
      uint32_t level = 0;
#pragma unroll
      for (int b = 0; b < 15; ++b) level += y > a.d4.m[b] ? 1u : 0u;
      const uint32_t c = (uint32_t)(a.d4.codes >> (4 * level)) & 15u;
      w[j / 8] |= c << (4 * (j % 8));
    }
    reinterpret_cast<uint2*>(dst)[u] = make_uint2(w[0], w[1]);
  }
}

struct KVReadArgs {
  KVPool pool;
  int64_t units;  // tokens * heads * 2 * dim / 16
  const int64_t* slots;
  uint16_t* k;
  uint16_t* v;
  Codebook cb;
  int* status;
};

// A thread reads back 16 elements of a row.
template <int KT>
__global__ __launch_bounds__(256) void kv_read_kernel(KVReadArgs a) {
  __shared__ __align__(16) float lut[16];
  if (KT == kKVNF4) {
    codebook_to_lds(lut, a.cb, threadIdx.x);
    __syncthreads();
  }
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= a.units) return;
  const uint32_t H = (uint32_t)a.pool.heads, units = (uint32_t)a.pool.dim / 16;
  const int64_t r = id / units;
  const uint32_t u = (uint32_t)(id - r * units);
  const int64_t ts = r / H;
  const uint32_t h = (uint32_t)(r - ts * H);
  const bool is_v = ts & 1;
  const int64_t tok = ts >> 1;
  const int64_t slot = a.slots[tok];
  u32x4 o[2] = {u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}};
  if (slot >= (a.pool.pages << a.pool.shift)) {
    if (u == 0 && h == 0) atomicOr(a.status, kStatusIndex);
  } else if (slot >= 0) {
    const int64_t mask = ((int64_t)1 << a.pool.shift) - 1;
    const int64_t row = (((slot >> a.pool.shift) * H + h) << a.pool.shift) + (slot & mask);
    const uint8_t* src = (is_v ? a.pool.v : a.pool.k) + row * kv_row_bytes(a.pool.type, a.pool.dim);
    if (KT == kKVBF16) {
      o[0] = reinterpret_cast<const u32x4*>(src)[2 * u];
      o[1] = reinterpret_cast<const u32x4*>(src)[2 * u + 1];
    } else {
      const float s = (is_v ? a.pool.vs : a.pool.ks)[row];
      float f[16];
      if (KT == kKVINT8) {
        const u32x4 w = reinterpret_cast<const u32x4*>(src)[u];
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] = (float)(int8_t)(w[j / 4] >> (8 * (j % 4))) * s;
      } else {
        const uint2 w = reinterpret_cast<const uint2*>(src)[u];
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] = lut[((j < 8 ? w.x : w.y) >> (4 * (j % 8))) & 15u] * s;
      }
#pragma unroll
      for (int q = 0; q < 2; ++q)
        o[q] = u32x4{pack_bf16x2(f[8 * q], f[8 * q + 1]), pack_bf16x2(f[8 * q + 2], f[8 * q + 3]),
                     pack_bf16x2(f[8 * q + 4], f[8 * q + 5]), pack_bf16x2(f[8 * q + 6], f[8 * q + 7])};
    }
  }
  uint16_t* dst = (is_v ? a.v : a.k) + (tok * H + h) * a.pool.dim;
  reinterpret_cast<u32x4*>(dst)[2 * u] = o[0];
  reinterpret_cast<u32x4*>(dst)[2 * u + 1] = o[1];
}

template <int KT, int LPR>
void write_rope(const KVWriteArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.rows + 256 / LPR - 1) / (256 / LPR)));
  if (!a.rope.table) hipLaunchKernelGGL((kv_write_kernel<KT, LPR, 0>), grid, dim3(256), 0, s, a);
  else if (!a.rope.interleaved) hipLaunchKernelGGL((kv_write_kernel<KT, LPR, 1>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((kv_write_kernel<KT, LPR, 2>), grid, dim3(256), 0, s, a);
}
template <int KT>
void write_lanes(const KVWriteArgs& a, hipStream_t s) {
  if (a.pool.dim <= 64) write_rope<KT, 4>(a, s);
  else if (a.pool.dim <= 128) write_rope<KT, 8>(a, s);
  else write_rope<KT, 16>(a, s);
}

}  // namespace

hipError_t launch_kv_write(const KVPool& pool, int64_t T, const HeadsView& k, const HeadsView& v,
                           const int64_t* slots, const RopeTable& rope, const Midpoints& mp, hipStream_t s) {
  KVWriteArgs a{};
  hipError_t e = hipSuccess;
  a.status = status_word(&e);
  if (!a.status) return e;
  a.pool = pool;
  a.k = k;
  a.v = v;
  a.rows = T * pool.heads * 2;
  a.slots = slots;
  a.rope = rope;
  for (int j = 0; j < 15; ++j) a.d4.m[j] = (float)mp.m[j];
  a.d4.codes = mp.codes;
  a.d4.zero_code = mp.zero_code;
  if (a.rows <= 0) return hipSuccess;
  KernelTimer kt_("kv_write_kernel", s);
  if (pool.type == kKVBF16) write_lanes<kKVBF16>(a, s);
  else if (pool.type == kKVINT8) write_lanes<kKVINT8>(a, s);
  else write_lanes<kKVNF4>(a, s);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KVPool& pool, int64_t T, const int64_t* slots, uint16_t* k, uint16_t* v,
                          const float table[16], hipStream_t s) {
  KVReadArgs a{};
  hipError_t e = hipSuccess;
  a.status = status_word(&e);
  if (!a.status) return e;
  a.pool = pool;
  a.units = T * pool.heads * 2 * (pool.dim / 16);
  a.slots = slots;
  a.k = k;
  a.v = v;
  for (int c = 0; c < 16; ++c) a.cb.c[c] = table[c];
  if (a.units <= 0) return hipSuccess;
  KernelTimer kt_("kv_read_kernel", s);
  const dim3 grid((unsigned)((a.units + 255) / 256));
  if (pool.type == kKVBF16) hipLaunchKernelGGL(kv_read_kernel<kKVBF16>, grid, dim3(256), 0, s, a);
  else if (pool.type == kKVINT8) hipLaunchKernelGGL(kv_read_kernel<kKVINT8>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(kv_read_kernel<kKVNF4>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace qlora
