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
// Both kernels move 2 bytes per element on the dense side, the row's codes and
// 4 bytes on the other.  Reading back and 8 and 16 bits are bound by memory:
// 4096 tokens of 32 heads of 128 read back from bf16 in 25 us (5.3 TB/s), int8
// 21 (4.9), NF4 20 (4.2), stored as bf16 34 (3.9, in scattered rows of 256
// bytes), int8 27 (3.7).  A 4-bit write is bound by its vector instructions:
// 2048 such tokens, rotated and stored in NF4, 15 us (43 MB; 34 with a
// comparison per boundary and a head per thread) issue 4.9 M of them, which take
// 19 k of the 31 k clocks that the kernel runs beyond an empty launch; its
// lookups and their conflicts take 3 k.  4001 tokens of 8
// heads, rotated, in int8: 8 us, 9973 read back 15 us (61 MB).
#include <cmath>
#include <mutex>

#include "common.hpp"
#include "device_state.hpp"
#include "kvcache.hpp"
#include "rope.hpp"
#include "timing.hpp"

namespace qlora {

namespace {

constexpr float kTinyRow = 1e-30f;

// How a level is decided: uniform bins of [-1, 1], each holding at most one
// boundary; entry = (the boundary, 2 where there is none; the codes below and
// above it).  kBins separates the boundaries of all three types by more than
// an fp32 estimate of the bin can err (checked on the host), so one read and
// one comparison give #{boundaries : y > m}.
constexpr int kBins = 127;
struct Bins {
  float m[kBins];
  uint8_t codes[kBins];
};

struct KVWriteArgs {
  KVPool pool;
  HeadsView k, v;
  int64_t T;
  int32_t groups;  // head groups of a token's row set
  const int64_t* slots;
  RopeTable rope;
  int* status;
};

// Largest of the LPR lanes of a row (LPR = 4, 8, 16), by lane exchanges inside
// the vector unit.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
  const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false);
  return y > x ? y : x;
}
template <int LPR>
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  x = dpp_max<0xB1>(x);                           // quad_perm [1,0,3,2]
  x = dpp_max<0x4E>(x);                           // quad_perm [2,3,0,1]
  if constexpr (LPR >= 8) x = dpp_max<0x141>(x);  // row_half_mirror
  if constexpr (LPR >= 16) x = dpp_max<0x140>(x); // row_mirror
  return x;
}

// LPR lanes per row, two pieces of 8 elements per lane: pieces that are turned
// against each other where the keys are rotated in the half layout, neighbours
// else.  A thread stores the same pieces of HB heads of a token, so a token's
// rotation is read once for all of them.
template <int KT, int LPR, int ROPE, int HB>
__global__ __launch_bounds__(256) void kv_write_kernel(KVWriteArgs a, Bins bins) {
  __shared__ float2 s_bin[KT == kKVNF4 ? kBins + 1 : 1];
  if (KT == kKVNF4) {
    const int t = threadIdx.x < kBins ? threadIdx.x : kBins - 1;
    if (threadIdx.x <= kBins) s_bin[threadIdx.x] = make_float2(bins.m[t], __uint_as_float(bins.codes[t]));
    __syncthreads();
  }
  const int64_t r = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  const int64_t ts = r / a.groups;
  const int h0 = (int)(r - ts * a.groups) * HB;
  const bool is_v = ts & 1;
  const int64_t tok = ts >> 1;
  if (tok >= a.T) return;  // the lanes of a row leave together
  const int H = a.pool.heads, u = threadIdx.x % LPR, D = a.pool.dim;
  const int64_t slot = a.slots[tok];
  if (slot < 0) return;
  if (slot >= (a.pool.pages << a.pool.shift)) {
    if (u == 0) atomicOr(a.status, kStatusIndex);
    return;
  }
  const bool mine = u * 16 < D;
  const bool turn = ROPE && !is_v && u * 16 < a.rope.rot;
  // The lane's pieces start at elements lo and hi.
  int lo = u * 16, hi = lo + 8;
  float cs[16];
  if (turn) {
    int64_t pos = a.rope.positions[tok];
    if (pos < 0 || pos >= a.rope.n) {
      if (u == 0) atomicOr(a.status, kStatusIndex);
      pos = 0;
    }
    if (ROPE == 1) {
      lo = u * 8;
      hi = lo + a.rope.rot / 2;
    }
    rope_row8(a.rope, pos, u * 8, 1.0f, cs);
  }
  const HeadsView& hv = is_v ? a.v : a.k;
  const uint16_t* src = hv.data + tok * hv.token_stride;
  u32x4 x[HB], y[HB];
#pragma unroll
  for (int i = 0; i < HB; ++i) {
    x[i] = y[i] = u32x4{0, 0, 0, 0};
    if (mine && h0 + i < H) {
      const uint16_t* p = src + (int64_t)(h0 + i) * hv.head_stride;
      x[i] = *reinterpret_cast<const u32x4*>(p + lo);
      y[i] = *reinterpret_cast<const u32x4*>(p + hi);
    }
  }
  const int64_t mask = ((int64_t)1 << a.pool.shift) - 1;
  const int64_t row_bytes = kv_row_bytes(a.pool.type, D);
#pragma unroll
  for (int i = 0; i < HB; ++i) {
    const int h = h0 + i;
    if (h >= H) return;
    float v[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = bf16_lo(x[i][q]);
      v[2 * q + 1] = bf16_hi(x[i][q]);
      v[8 + 2 * q] = bf16_lo(y[i][q]);
      v[8 + 2 * q + 1] = bf16_hi(y[i][q]);
    }
    if (turn) {
#pragma unroll
      for (int q = 0; q < 8; ++q) rope_pair(v[ROPE == 1 ? q : 2 * q], v[ROPE == 1 ? 8 + q : 2 * q + 1], cs[2 * q], cs[2 * q + 1]);
    }
    const int64_t row = (((slot >> a.pool.shift) * H + h) << a.pool.shift) + (slot & mask);
    uint8_t* dst = (is_v ? a.pool.v : a.pool.k) + row * row_bytes;
    if constexpr (KT == kKVBF16) {
      if (mine) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
          *reinterpret_cast<u32x4*>(dst + 2 * (q ? hi : lo)) =
              u32x4{pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                    pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7])};
      }
    } else {
      // The row's largest magnitude, as integers: NaN > infinity > every number.
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t b = __float_as_uint(v[j]) & 0x7FFFFFFFu;
        top = b > top ? b : top;
      }
      top = row_max<LPR>(top);
      const float t = __uint_as_float(top);
      const bool fine = t >= kTinyRow;
      const float unit = fine ? 1.0f / t : 0.0f;
      if (u == 0) {
        float s = KT == kKVINT8 ? t * (float)(1.0 / 127.0) : t;
        if (!fine) s = 0.0f;
        if (top >= 0x7F800000u) s = __uint_as_float(0x7FC00000u);
        (is_v ? a.pool.vs : a.pool.ks)[row] = s;
      }
      if constexpr (KT == kKVINT8) {
        const float m = unit * 127.0f;
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          w[q] = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float c = __builtin_amdgcn_fmed3f(rintf(v[4 * q + j] * m), -127.0f, 127.0f);
            w[q] |= ((uint32_t)(int)c & 0xFFu) << (8 * j);
          }
        }
        if (mine) {
          *reinterpret_cast<uint2*>(dst + lo) = make_uint2(w[0], w[1]);
          *reinterpret_cast<uint2*>(dst + hi) = make_uint2(w[2], w[3]);
        }
      } else {
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float e = v[j] * unit;
          // NaN and out-of-range products (a row that is no numbers) land in a bin too.
          const int bin = (int)__builtin_amdgcn_fmed3f(__builtin_fmaf(e, 0.5f * kBins, 0.5f * kBins), 0.0f, (float)(kBins - 1));
          const float2 d = s_bin[bin];
          w[j / 8] |= ((__float_as_uint(d.y) >> (e > d.x ? 4 : 0)) & 15u) << (4 * (j % 8));
        }
        if (mine) {
          *reinterpret_cast<uint32_t*>(dst + lo / 2) = w[0];
          *reinterpret_cast<uint32_t*>(dst + hi / 2) = w[1];
        }
      }
    }
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

template <int KT, int LPR, int HB>
void write_rope(KVWriteArgs a, const Bins& bins, hipStream_t s) {
  a.groups = (a.pool.heads + HB - 1) / HB;
  const int64_t rows = a.T * 2 * a.groups;
  const dim3 grid((unsigned)((rows + 256 / LPR - 1) / (256 / LPR)));
  if (!a.rope.table) hipLaunchKernelGGL((kv_write_kernel<KT, LPR, 0, HB>), grid, dim3(256), 0, s, a, bins);
  else if (!a.rope.interleaved) hipLaunchKernelGGL((kv_write_kernel<KT, LPR, 1, HB>), grid, dim3(256), 0, s, a, bins);
  else hipLaunchKernelGGL((kv_write_kernel<KT, LPR, 2, HB>), grid, dim3(256), 0, s, a, bins);
}
template <int KT, int LPR>
void write_heads(const KVWriteArgs& a, const Bins& bins, hipStream_t s) {
  if (kv_write_heads(a.T, a.pool.heads, a.pool.dim) == 4) write_rope<KT, LPR, 4>(a, bins, s);
  else write_rope<KT, LPR, 1>(a, bins, s);
}
template <int KT>
void write_lanes(const KVWriteArgs& a, const Bins& bins, hipStream_t s) {
  const int lanes = kv_write_lanes(a.pool.dim);
  if (lanes == 4) write_heads<KT, 4>(a, bins, s);
  else if (lanes == 8) write_heads<KT, 8>(a, bins, s);
  else write_heads<KT, 16>(a, bins, s);
}

// The bins of a type; false if kBins does not separate its boundaries.
bool make_kv_bins(const Midpoints& mp, Bins* out) {
  for (int b = 0; b < kBins; ++b) {
    const double lo = -1.0 + b * (2.0 / kBins), hi = lo + 2.0 / kBins;
    uint32_t below = 0, inside = 0;
    out->m[b] = 2.0f;
    for (int j = 0; j < 15; ++j) {
      const double m = (float)mp.m[j];  // +inf past the type's last
      if (m < lo) ++below;
      else if (m < hi) {
        ++inside;
        out->m[b] = (float)m;
      }
      if (std::fabs(m - lo) < 1e-5 || std::fabs(m - hi) < 1e-5) return false;
    }
    if (inside > 1) return false;
    out->codes[b] = (uint8_t)(level_code(mp, below) | (level_code(mp, below + 1 < 16 ? below + 1 : 15) << 4));
  }
  return true;
}

// The same, built once per type.
bool kv_bins(int type, const Midpoints& mp, Bins* out) {
  static std::once_flag once[3];
  static Bins bins[3];
  static bool good[3];
  const int i = type - kKVNF4;
  std::call_once(once[i], [&] { good[i] = make_kv_bins(mp, &bins[i]); });
  *out = bins[i];
  return good[i];
}

}  // namespace

hipError_t launch_kv_write(const KVPool& pool, int64_t T, const HeadsView& k, const HeadsView& v,
                           const int64_t* slots, const RopeTable& rope, const Midpoints& mp, hipStream_t s) {
  KVWriteArgs a{};
  Bins bins{};
  hipError_t e = hipSuccess;
  a.status = status_word(&e);
  if (!a.status) return e;
  if (pool.type >= kKVNF4 && !kv_bins(pool.type, mp, &bins)) return hipErrorInvalidValue;  // no shipped type
  a.pool = pool;
  a.k = k;
  a.v = v;
  a.T = T;
  a.slots = slots;
  a.rope = rope;
  KernelTimer kt_("kv_write_kernel", s);
  if (pool.type == kKVBF16) write_lanes<kKVBF16>(a, bins, s);
  else if (pool.type == kKVINT8) write_lanes<kKVINT8>(a, bins, s);
  else write_lanes<kKVNF4>(a, bins, s);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KVPool& pool, int64_t T, const int64_t* slots, uint16_t* k, uint16_t* v,
                          const float table[16], hipStream_t s) {
  KVReadArgs a{};
  hipError_t e = hipSuccess;
  a.status = status_word(&e);
  if (!a.status) return e;
  a.pool = pool;
  a.units = kv_read_threads(T, pool.heads, pool.dim);
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
