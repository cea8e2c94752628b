// Global gradient norm over many tensors, and clipping (QLoRA project page,
// challenges: gradient clipping keeps training stable), for gfx950.
//
//   |g| = sqrt(sum over all tensors of g_i^2),
//   c = min(1, max_norm / (|g| + 1e-6)),   out_i = c g_i
//
// The adapters of a model are hundreds of small tensors.  Their addresses and
// lengths come as kernel arguments, so that nothing has to be copied to the
// device and a captured call holds all it needs: up to kSetMax of them go to the
// two kernels directly, more are first written to the workspace by launches that
// do nothing else.  Both kernels see one row of chunks of kChunk values over all
// tensors, and each workgroup takes a run of neighbours: it looks its first
// tensor up and then only steps on.  Squares are summed in fp64; each workgroup
// leaves one partial, and every workgroup of the second kernel adds the partials
// in the same order, so the result does not depend on timing.  The second kernel walks its
// run backwards: what the first read last is still in the caches.
//
// Bound by memory: two reads and a write.  448 gradients of 216 M bf16 values:
// 242 us, 5.4 TB/s of 1.3 GB.
#include "common.hpp"
#include "timing.hpp"
#include "train.hpp"

namespace qlora {

namespace {
constexpr int kSetMax = 112;       // 32 bytes each: the arguments stay below 4 KB
constexpr int kThreads = 256;
constexpr int kChunk = 16384;      // values
constexpr int kGridMax = 2048;     // workgroups (and partials)

struct SetEntry {
  const void* grad;
  void* out;
  int64_t n;
  uint32_t first;  // chunk at which the tensor starts
  uint32_t kind;   // bit 0: grad is fp32, bit 1: out is fp32
};
struct SetArgs {
  SetEntry e[kSetMax];
};
// All tensors: entries in the workspace, or (null) in the arguments.
struct GradSet {
  const SetEntry* e;
  uint32_t chunks;  // of all tensors
  int32_t count;
};

// The tensor of chunk c: the last that starts at or before it.
__device__ __forceinline__ int tensor_of(const SetEntry* e, int count, uint32_t c) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (e[mid].first <= c) lo = mid;
    else hi = mid - 1;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}
// This workgroup's run of chunks.
struct Run {
  uint32_t begin, end;
};
__device__ __forceinline__ Run run_of(uint32_t chunks) {
  const uint32_t each = (chunks + gridDim.x - 1) / gridDim.x, b = blockIdx.x * each;
  return Run{b < chunks ? b : chunks, b + each < chunks ? b + each : chunks};
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

// Eight values of a thread as they are stored.  Where neither side is fp32 they
// are neighbours; otherwise (SPLIT) two groups of four, kThreads groups apart, so
// that a wave's access of 16 bytes a lane is without gaps on the wide side too (with
// gaps, marked stores of fp32 took 96 us instead of 66 at 128 MiB).
template <bool WIDE>
struct Raw8 {
  u32x4 u[WIDE ? 2 : 1];
};
using u32v2 = __attribute__((ext_vector_type(2))) unsigned int;
using u32v4 = __attribute__((ext_vector_type(4))) unsigned int;
// Byte offset of half h of group i (of eight) of a thread's.
template <bool WIDE, bool SPLIT>
__device__ __forceinline__ int half_at(int i, int h) {
  return (SPLIT ? (8 * i + 4 * h) * kThreads + 4 * (int)threadIdx.x : 8 * (i * kThreads + (int)threadIdx.x) + 4 * h) * (WIDE ? 4 : 2);
}
// (Buffer views: what lies past a chunk's end reads as zero and is not written,
// without a branch that would hold the next load back.)  NT: marked as used once
// (the instruction's nt bit).
template <bool WIDE, bool SPLIT, bool NT>
__device__ __forceinline__ Raw8<WIDE> load8(rsrc_t r, int i) {
  constexpr int aux = NT ? 2 : 0;
  Raw8<WIDE> x;
  if constexpr (WIDE) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      x.u[h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, half_at<true, SPLIT>(i, h), 0, aux));
  } else if constexpr (SPLIT) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32v2 v = __builtin_bit_cast(u32v2, __builtin_amdgcn_raw_buffer_load_b64(r, half_at<false, true>(i, h), 0, aux));
      x.u[0][2 * h] = v[0];
      x.u[0][2 * h + 1] = v[1];
    }
  } else {
    x.u[0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, half_at<false, false>(i, 0), 0, aux));
  }
  return x;
}
template <bool WIDE>
__device__ __forceinline__ void values(const Raw8<WIDE>& r, float (&v)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (WIDE) {
      v[q] = __uint_as_float(r.u[0][q]);
      v[4 + q] = __uint_as_float(r.u[1][q]);
    } else {
      v[2 * q] = bf16_lo(r.u[0][q]);
      v[2 * q + 1] = bf16_hi(r.u[0][q]);
    }
  }
}
template <bool WIDE>
__device__ __forceinline__ float load1(const void* base, int64_t i) {
  if constexpr (WIDE) return static_cast<const float*>(base)[i];
  else return bf16_to_f32(static_cast<const uint16_t*>(base)[i]);
}
template <bool WIDE, bool SPLIT, bool NT>
__device__ __forceinline__ void store8(rsrc_t r, int i, const float (&v)[8]) {
  constexpr int aux = NT ? 2 : 0;
  if constexpr (WIDE) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      __builtin_amdgcn_raw_buffer_store_b128(u32v4{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]), __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])},
                                             r, half_at<true, SPLIT>(i, h), 0, aux);
  } else {
    const uint32_t w[4] = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    if constexpr (SPLIT) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        __builtin_amdgcn_raw_buffer_store_b64(u32v2{w[2 * h], w[2 * h + 1]}, r, half_at<false, true>(i, h), 0, aux);
    } else {
      __builtin_amdgcn_raw_buffer_store_b128(u32v4{w[0], w[1], w[2], w[3]}, r, half_at<false, false>(i, 0), 0, aux);
    }
  }
}
// A view of n values from value i0 on.
template <bool WIDE>
__device__ __forceinline__ rsrc_t view(const void* base, int64_t i0, int n) {
  return make_rsrc(static_cast<const char*>(base) + i0 * (WIDE ? 4 : 2), (int64_t)n * (WIDE ? 4 : 2));
}
template <bool WIDE>
__device__ __forceinline__ void store1(void* base, int64_t i, float v) {
  if constexpr (WIDE) static_cast<float*>(base)[i] = v;
  else static_cast<uint16_t*>(base)[i] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFF);
}

__device__ __forceinline__ bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kVecs = kChunk / (8 * kThreads);  // groups of eight values of a thread in a whole chunk

// The squares of eight values.  (Summed in fp32, eight at a time, where they are in
// its range, they take as long: the norm of 226 M values, in fp32 and in fp64, bf16
// 88.1 and 88.4 us, fp32 162.6 and 161.1; of 67 M fp32 values 43.9 and 45.0.)
__device__ __forceinline__ double squares8(const float (&v)[8]) {
  double x = 0.0;
#pragma unroll
  for (int q = 0; q < 8; ++q) x += square(v[q]);
  return x;
}

// Tensors that start on 16 bytes go eight values at a time, others (views at
// odd places) one by one.
template <bool WIDE>
__device__ __forceinline__ double chunk_squares(const void* g, int64_t i0, int n) {
  double acc = 0.0;
  const int tid = threadIdx.x;
  int done = 0;
  if (on16(g)) {
    done = n & ~7;
    const rsrc_t in = view<WIDE>(g, i0, done);
    Raw8<WIDE> r[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) r[k] = load8<WIDE, WIDE, false>(in, k);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      float v[8];
      values<WIDE>(r[k], v);
      acc += squares8(v);
    }
  }
#pragma unroll 8
  for (int i = done + tid; i < n; i += kThreads) acc += square(load1<WIDE>(g, i0 + i));
  return acc;
}

// (`out` may be `g` itself: a thread reads what it writes, and a chunk is read
// before it is written.)
template <bool WIDE, bool OUT_WIDE, bool NT>
__device__ __forceinline__ void chunk_scale(const void* g, void* out, int64_t i0, int n, float c) {
  const int tid = threadIdx.x;
  int done = 0;
  if (on16(g) && on16(out)) {
    done = n & ~7;
    const rsrc_t in = view<WIDE>(g, i0, done), to = view<OUT_WIDE>(out, i0, done);
    Raw8<WIDE> r[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) r[k] = load8<WIDE, WIDE || OUT_WIDE, NT>(in, k);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      float v[8];
      values<WIDE>(r[k], v);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] *= c;
      store8<OUT_WIDE, WIDE || OUT_WIDE, NT>(to, k, v);
    }
  }
  for (int i = done + tid; i < n; i += kThreads) store1<OUT_WIDE>(out, i0 + i, load1<WIDE>(g, i0 + i) * c);
}
}  // namespace

__global__ __launch_bounds__(128) void grads_table_kernel(SetArgs args, SetEntry* out, int n) {
  if ((int)threadIdx.x < n) out[threadIdx.x] = args.e[threadIdx.x];
}

// partial[b] = the squares of this workgroup's chunks.
__global__ __launch_bounds__(kThreads) void grads_sumsq_kernel(GradSet s, SetArgs args, double* __restrict__ partial) {
  __shared__ double red[4];
  const SetEntry* const e = s.e ? s.e : args.e;
  const Run run = run_of(s.chunks);
  double acc = 0.0;
  if (run.begin < run.end) {
    int i = tensor_of(e, s.count, run.begin);
    for (uint32_t c = run.begin; c < run.end; ++c) {
      while (i + 1 < s.count && e[i + 1].first <= c) ++i;
      const int64_t i0 = (int64_t)(c - e[i].first) * kChunk;
      const int n = (int)(e[i].n - i0 < kChunk ? e[i].n - i0 : kChunk);
      acc += e[i].kind & 1 ? chunk_squares<true>(e[i].grad, i0, n) : chunk_squares<false>(e[i].grad, i0, n);
    }
  }
  const double sum = block_sum(acc, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// From kStreamBytes of gradients on the second kernel marks its accesses as used
// once, so that they leave those gradients in the last cache that it still has to
// read.  Clipping into other tensors and, in parentheses, writing the
// gradients, clipping them in place and reading them, bf16, us without and with the
// mark: 43 (82) and 39 (82) at 64 MiB, 70 (157) and 68 (163) at 128, 112 (248) and
// 97 (245) at 192, 159 (359) and 129 (335) at 256, 317 (725) and 273 (690) at 512.
template <bool NT>
__global__ __launch_bounds__(kThreads) void grads_scale_kernel(GradSet s, SetArgs args,
                                                               const double* __restrict__ partial, int nparts,
                                                               float max_norm, float* norm_out) {
  __shared__ double red[4];
  double x = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kThreads) x += partial[i];
  const double norm = sqrt(block_sum(x, red));
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm_out) *norm_out = (float)norm;
  if (!(max_norm > 0.0f)) return;
  const double cc = (double)max_norm / (norm + 1e-6);
  const float c = cc >= 1.0 ? 1.0f : (float)cc;  // a norm that is no number gives a coefficient that is none
  const SetEntry* const e = s.e ? s.e : args.e;
  const Run run = run_of(s.chunks);
  if (run.begin >= run.end) return;
  int i = tensor_of(e, s.count, run.end - 1);
  for (uint32_t ch = run.end; ch-- > run.begin;) {
    while (e[i].first > ch) --i;
    if (!e[i].out || (c == 1.0f && e[i].out == e[i].grad)) continue;
    const int64_t i0 = (int64_t)(ch - e[i].first) * kChunk;
    const int n = (int)(e[i].n - i0 < kChunk ? e[i].n - i0 : kChunk);
    switch (e[i].kind & 3) {
      case 0: chunk_scale<false, false, NT>(e[i].grad, e[i].out, i0, n, c); break;
      case 1: chunk_scale<true, false, NT>(e[i].grad, e[i].out, i0, n, c); break;
      case 2: chunk_scale<false, true, NT>(e[i].grad, e[i].out, i0, n, c); break;
      default: chunk_scale<true, true, NT>(e[i].grad, e[i].out, i0, n, c); break;
    }
  }
}

size_t clip_grads_workspace_bytes(int count) {
  return sizeof(double) * kGridMax + (count > kSetMax ? sizeof(SetEntry) * (size_t)count : 0);
}

hipError_t launch_clip_grads(int count, const GradTensor* g, float max_norm, float* norm_out, void* ws,
                             hipStream_t s) {
  double* partial = static_cast<double*>(ws);
  SetEntry* table = reinterpret_cast<SetEntry*>(partial + kGridMax);
  SetArgs args;
  uint32_t at = 0;
  int64_t bytes = 0;
  for (int i = 0; i < count; ++i) {
    bytes += g[i].n * (g[i].wide ? 4 : 2);
    args.e[i % kSetMax] = SetEntry{g[i].grad, g[i].out, g[i].n, at, (g[i].wide ? 1u : 0u) | (g[i].out_wide ? 2u : 0u)};
    at += (uint32_t)((g[i].n + kChunk - 1) / kChunk);
    const int filled = i % kSetMax + 1;
    if (count > kSetMax && (filled == kSetMax || i + 1 == count)) {
      KernelTimer kt_("grads_table_kernel", s);
      hipLaunchKernelGGL(grads_table_kernel, dim3(1), dim3(128), 0, s, args, table + (i + 1 - filled), filled);
      hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  const GradSet set{count > kSetMax ? table : nullptr, at, count};
  const int grid = at < 1 ? 1 : at < (uint32_t)kGridMax ? (int)at : kGridMax;
  {
    KernelTimer kt_("grads_sumsq_kernel", s);
    hipLaunchKernelGGL(grads_sumsq_kernel, dim3(grid), dim3(kThreads), 0, s, set, args, partial);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  {
    KernelTimer kt_("grads_scale_kernel", s);
    const dim3 grid2(max_norm > 0.0f ? grid : 1);
    if (bytes >= kStreamBytes)
      hipLaunchKernelGGL(grads_scale_kernel<true>, grid2, dim3(kThreads), 0, s, set, args, partial, grid, max_norm, norm_out);
    else
      hipLaunchKernelGGL(grads_scale_kernel<false>, grid2, dim3(kThreads), 0, s, set, args, partial, grid, max_norm, norm_out);
  }
  return hipGetLastError();
}

}  // namespace qlora
