// Global gradient norm over many tensors, and clipping (QLoRA project page,
// challenges: gradient clipping keeps training stable), for gfx950.
//
//   |g| = sqrt(sum over all tensors of g_i^2),
//   c = min(1, max_norm / (|g| + 1e-6)),   out_i = c g_i
//
// The adapters of a model are hundreds of small tensors.  Their addresses and
// lengths travel as kernel arguments, up to kSetMax to a launch, so that
// nothing has to be copied to the device first and a captured call holds all
// it needs.  A launch has one grid over all its tensors, cut into chunks of
// kChunk values; the workgroups walk the chunks with a fixed stride.  Squares
// are exact in fp64 and summed there (the product of two fp32 values has 48
// bits); each workgroup leaves one fp64 partial, and every workgroup of the
// second launch adds the partials in the same order, so the result does not
// depend on timing.
#include "common.hpp"
#include "timing.hpp"
#include "train.hpp"

namespace qlora {

namespace {
constexpr int kSetMax = 112;       // 32 bytes each: the arguments stay below 4 KB
constexpr int kThreads = 256;
constexpr int kChunk = 16384;      // values
constexpr int kGridMax = 1024;     // workgroups (and partials) of a launch

struct SetEntry {
  const void* grad;
  void* out;
  int64_t n;
  uint32_t first;  // chunk at which the tensor starts
  uint32_t kind;   // bit 0: grad is fp32, bit 1: out is fp32
};
struct GradSet {
  SetEntry e[kSetMax];
  uint32_t chunks;  // of all tensors
  int32_t count;
};

// The tensor of chunk c: the last that starts at or before it.
__device__ __forceinline__ int tensor_of(const GradSet& s, uint32_t c) {
  int lo = 0, hi = s.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.e[mid].first <= c) lo = mid;
    else hi = mid - 1;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

__device__ __forceinline__ double block_sum(double x, double* red) {
#pragma unroll
  for (int off = 32; off; off >>= 1) x += __shfl_xor(x, off, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

__device__ __forceinline__ double square(float x) { return (double)x * (double)x; }

// Eight consecutive values as fp32.
template <bool WIDE>
__device__ __forceinline__ void load8(const void* base, int64_t i, float (&v)[8]) {
  if constexpr (WIDE) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const u32x4 u = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + i);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = bf16_lo(u[q]);
      v[2 * q + 1] = bf16_hi(u[q]);
    }
  }
}
template <bool WIDE>
__device__ __forceinline__ float load1(const void* base, int64_t i) {
  if constexpr (WIDE) return static_cast<const float*>(base)[i];
  else return bf16_to_f32(static_cast<const uint16_t*>(base)[i]);
}
template <bool WIDE>
__device__ __forceinline__ void store8(void* base, int64_t i, const float (&v)[8]) {
  if constexpr (WIDE) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + i) =
        u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  }
}
template <bool WIDE>
__device__ __forceinline__ void store1(void* base, int64_t i, float v) {
  if constexpr (WIDE) static_cast<float*>(base)[i] = v;
  else static_cast<uint16_t*>(base)[i] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFF);
}

__device__ __forceinline__ bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kVecs = kChunk / (8 * kThreads);  // groups of eight values of a thread in a whole chunk
constexpr int kBatch = 4;                       // of them on their way at a time

// Tensors that start on 16 bytes go eight values at a time, others (views at
// odd places) one by one.
template <bool WIDE>
__device__ __forceinline__ double chunk_squares(const void* g, int64_t i0, int n) {
  double acc = 0.0;
  const int tid = threadIdx.x;
  int done = 0;
  if (on16(g)) {
    done = n & ~7;
#pragma unroll
    for (int k0 = 0; k0 < kVecs; k0 += kBatch) {
      float v[kBatch][8];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = ((k0 + k) * kThreads + tid) * 8;
        if (i < done) load8<WIDE>(g, i0 + i, v[k]);
        else
#pragma unroll
          for (int q = 0; q < 8; ++q) v[k][q] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int q = 0; q < 8; ++q) acc += square(v[k][q]);
    }
  }
#pragma unroll 8
  for (int i = done + tid; i < n; i += kThreads) acc += square(load1<WIDE>(g, i0 + i));
  return acc;
}

// (`out` may be `g` itself: a thread reads what it writes, and a batch is read
// before it is written.)
template <bool WIDE, bool OUT_WIDE>
__device__ __forceinline__ void chunk_scale(const void* g, void* out, int64_t i0, int n, float c) {
  const int tid = threadIdx.x;
  int done = 0;
  if (on16(g) && on16(out)) {
    done = n & ~7;
#pragma unroll
    for (int k0 = 0; k0 < kVecs; k0 += kBatch) {
      float v[kBatch][8];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = ((k0 + k) * kThreads + tid) * 8;
        if (i < done) load8<WIDE>(g, i0 + i, v[k]);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = ((k0 + k) * kThreads + tid) * 8;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[k][q] *= c;
        if (i < done) store8<OUT_WIDE>(out, i0 + i, v[k]);
      }
    }
  }
  for (int i = done + tid; i < n; i += kThreads) store1<OUT_WIDE>(out, i0 + i, load1<WIDE>(g, i0 + i) * c);
}
}  // namespace

// partial[b] = the squares of this workgroup's chunks.
__global__ __launch_bounds__(kThreads) void grads_sumsq_kernel(GradSet s, double* __restrict__ partial) {
  __shared__ double red[4];
  double acc = 0.0;
  for (uint32_t c = blockIdx.x; c < s.chunks; c += gridDim.x) {
    const SetEntry& e = s.e[tensor_of(s, c)];
    const int64_t i0 = (int64_t)(c - e.first) * kChunk;
    const int n = (int)(e.n - i0 < kChunk ? e.n - i0 : kChunk);
    acc += e.kind & 1 ? chunk_squares<true>(e.grad, i0, n) : chunk_squares<false>(e.grad, i0, n);
  }
  const double sum = block_sum(acc, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__global__ __launch_bounds__(kThreads) void grads_scale_kernel(GradSet s, const double* __restrict__ partial,
                                                               int nparts, float max_norm, float* norm_out) {
  __shared__ double red[4];
  double x = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kThreads) x += partial[i];
  const double norm = sqrt(block_sum(x, red));
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm_out) *norm_out = (float)norm;
  if (!(max_norm > 0.0f)) return;
  const double cc = (double)max_norm / (norm + 1e-6);
  const float c = cc >= 1.0 ? 1.0f : (float)cc;  // a norm that is no number gives a coefficient that is none
  for (uint32_t ch = blockIdx.x; ch < s.chunks; ch += gridDim.x) {
    const SetEntry& e = s.e[tensor_of(s, ch)];
    if (!e.out || (c == 1.0f && e.out == e.grad)) continue;
    const int64_t i0 = (int64_t)(ch - e.first) * kChunk;
    const int n = (int)(e.n - i0 < kChunk ? e.n - i0 : kChunk);
    switch (e.kind & 3) {
      case 0: chunk_scale<false, false>(e.grad, e.out, i0, n, c); break;
      case 1: chunk_scale<true, false>(e.grad, e.out, i0, n, c); break;
      case 2: chunk_scale<false, true>(e.grad, e.out, i0, n, c); break;
      default: chunk_scale<true, true>(e.grad, e.out, i0, n, c); break;
    }
  }
}

namespace {
int set_launches(int count) { return (count + kSetMax - 1) / kSetMax; }

GradSet make_set(int count, const GradTensor* g) {
  GradSet s;
  s.count = count;
  uint32_t at = 0;
  for (int i = 0; i < count; ++i) {
    s.e[i] = SetEntry{g[i].grad, g[i].out, g[i].n, at, (g[i].wide ? 1u : 0u) | (g[i].out_wide ? 2u : 0u)};
    at += (uint32_t)((g[i].n + kChunk - 1) / kChunk);
  }
  s.chunks = at;
  return s;
}
int set_grid(const GradSet& s) { return s.chunks < 1 ? 1 : s.chunks < (uint32_t)kGridMax ? (int)s.chunks : kGridMax; }
}  // namespace

size_t clip_grads_workspace_bytes(int count) {
  return sizeof(double) * (size_t)kGridMax * (size_t)(count > 0 ? set_launches(count) : 1);
}

hipError_t launch_clip_grads(int count, const GradTensor* g, float max_norm, float* norm_out, void* ws,
                             hipStream_t s) {
  double* partial = static_cast<double*>(ws);
  int parts = 0;
  for (int i = 0; i == 0 || i < count; i += kSetMax) {
    const GradSet set = make_set(count - i < kSetMax ? count - i : kSetMax, g + i);
    const int grid = set_grid(set);
    KernelTimer kt_("grads_sumsq_kernel", s);
    hipLaunchKernelGGL(grads_sumsq_kernel, dim3(grid), dim3(kThreads), 0, s, set, partial + parts);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    parts += grid;
  }
  for (int i = 0; i == 0 || i < count; i += kSetMax) {
    const GradSet set = make_set(count - i < kSetMax ? count - i : kSetMax, g + i);
    const bool only_norm = !(max_norm > 0.0f);
    KernelTimer kt_("grads_scale_kernel", s);
    hipLaunchKernelGGL(grads_scale_kernel, dim3(only_norm ? 1 : set_grid(set)), dim3(kThreads), 0, s, set, partial,
                       parts, max_norm, i == 0 ? norm_out : nullptr);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (only_norm) break;
  }
  return hipSuccess;
}

}  // namespace qlora
