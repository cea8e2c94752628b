// Rotary positions, the paged key/value cache and attention over it: host
// structures shared by the kernels' launchers and the C entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qlora {

struct Midpoints;

// Element types of a cache (values of qlora_kv_type).
enum KVType { kKVBF16 = 0, kKVINT8 = 1, kKVNF4 = 2, kKVINT4 = 3, kKVFP4 = 4, kKVTypes = 5 };

// [tokens, heads, dim] bf16 with the dims of a head contiguous.
struct HeadsView {
  uint16_t* data;
  int64_t token_stride, head_stride;  // elements
  int32_t heads;
};

// Page p holds, head by head, its page_size rows of `dim` elements; row
// (p, h, s) is number ((p * heads + h) << shift) + s of codes and scales.
struct KVPool {
  uint8_t* k;
  uint8_t* v;
  float* ks;  // one fp32 scale per row (null for bf16)
  float* vs;
  int32_t type, heads, dim, shift;  // page_size = 1 << shift
  int64_t pages;
};

// Bytes of a row's codes.
__host__ __device__ __forceinline__ int64_t kv_row_bytes(int type, int dim) {
  return type == kKVBF16 ? 2 * dim : type == kKVINT8 ? dim : dim / 2;
}

// A launch counts its threads in 32 bits along an axis: one of more comes back
// as an error, or silently as what is left of the count.  `threads` in whole
// workgroups of up to 512 stays below that.
inline bool grid_fits(int64_t threads) { return threads <= (int64_t(1) << 32) - 512; }
// Threads of the rotation, of its table, and of the cache's two kernels (see
// their launchers).
inline int64_t rope_threads(int64_t tokens, int64_t heads, int32_t dim) { return tokens * heads * (dim / 16); }
inline int64_t rope_table_threads(int64_t positions, int32_t rot) { return positions * (rot / 2); }
inline int kv_write_lanes(int32_t dim) { return dim <= 64 ? 4 : dim <= 128 ? 8 : 16; }  // of a row
inline int64_t kv_read_threads(int64_t tokens, int64_t heads, int32_t dim) { return tokens * heads * 2 * (dim / 16); }
// Heads that a thread of the cache write takes: four once that leaves enough
// workgroups.
inline int kv_write_heads(int64_t tokens, int64_t heads, int32_t dim) {
  return tokens * 2 * heads * kv_write_lanes(dim) >= 4 * 256 * 1024 ? 4 : 1;
}
inline int64_t kv_write_threads(int64_t tokens, int64_t heads, int32_t dim) {
  const int n = kv_write_heads(tokens, heads, dim);
  return tokens * 2 * ((heads + n - 1) / n) * kv_write_lanes(dim);
}

// A cos/sin table and the positions that pick its rows; table = null: no
// rotation.
struct RopeTable {
  const float* table;  // [n][rot / 2][2]
  int64_t n;
  const int32_t* positions;  // [tokens]
  int32_t rot, interleaved;
};

struct RopeTableArgs {
  int64_t n;
  int32_t rot, scaling;
  double base, factor, original, low, high, amplitude;
};
hipError_t launch_rope_table(const RopeTableArgs& a, float* table, hipStream_t s);

hipError_t launch_rope(int64_t T, int32_t dim, const RopeTable& t, bool inverse, const HeadsView& q,
                       const HeadsView& q_out, const HeadsView& k, const HeadsView& k_out, hipStream_t s);

hipError_t launch_kv_write(const KVPool& pool, int64_t T, const HeadsView& k, const HeadsView& v,
                           const int64_t* slots, const RopeTable& rope, const Midpoints& mp, hipStream_t s);
hipError_t launch_kv_read(const KVPool& pool, int64_t T, const int64_t* slots, uint16_t* k, uint16_t* v,
                          const float table[16], hipStream_t s);

struct AttendProblem {
  KVPool pool;
  HeadsView q;
  int64_t tokens;
  int32_t batch;
  const int32_t* pages;  // [batch][width]
  int64_t width;
  const int32_t* starts;   // [batch + 1]
  const int32_t* lengths;  // [batch]
  int32_t max_new, max_len;
  float scale;
  int32_t causal, window;
  uint16_t* out;
  float* lse;  // may be null
};
size_t attend_workspace_bytes(const AttendProblem& p);
// False when a launch of this problem would exceed a grid or index limit.
bool attend_fits(const AttendProblem& p);
hipError_t launch_attend(const AttendProblem& p, const float table[16], void* ws, hipStream_t s);

}  // namespace qlora
