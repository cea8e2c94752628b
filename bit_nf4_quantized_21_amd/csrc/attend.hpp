// Attention over the paged cache: what its kernels share on the device.
#pragma once

#include "common.hpp"
#include "device_state.hpp"
#include "kvcache.hpp"

namespace qlora {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMaxChunk = 16384;   // keys of a split (streaming): bounds its page list in LDS
constexpr int kListKeys = 8192;    // keys that a tile workgroup's page list in LDS covers at a time

struct AttendArgs {
  KVPool pool;
  HeadsView q;
  int64_t tokens;
  const int32_t* pages;
  int64_t width;
  const int32_t* starts;
  const int32_t* lengths;
  int32_t batch, group, max_new, max_len;
  float scale2;  // scale * log2(e)
  int32_t causal, window;
  uint16_t* out;
  float* lse;
  float* part_o;   // [splits][tokens][q heads][dim]
  float* part_ml;  // [splits][tokens][q heads][2]
  int32_t splits, chunk, tiles;  // keys per split (a multiple of 128), row tiles
  uint32_t levels[16];  // 4-bit cache: bf16 level (low half) and what it misses of the value (high half)
  float values[16];     // 4-bit cache: the levels in fp32
  float unit;           // value = level * unit * scale of the row
  int* status;
};

// Quotient of values that are the same on every lane, in a scalar register
// (the division itself runs on vector units).
__device__ __forceinline__ int uniform_div(int a, int b) {
  return __builtin_amdgcn_readfirstlane((int)((uint32_t)a / (uint32_t)b));
}

// A sequence's tokens and length, held inside what the caller's sizes allow.
struct Seq {
  int64_t first;  // row of its first new token
  int n, len;
  bool bad;
};
__device__ __forceinline__ Seq load_seq(const AttendArgs& a, int b) {
  // (Uniform: kept in scalar registers.)
  int64_t s0 = __builtin_amdgcn_readfirstlane(a.starts[b]), s1 = __builtin_amdgcn_readfirstlane(a.starts[b + 1]);
  int64_t len = __builtin_amdgcn_readfirstlane(a.lengths[b]);
  Seq q;
  // The sequences cover the tokens: a row outside of them would not be written.
  q.bad = (b == 0 && s0 != 0) || (b == a.batch - 1 && s1 != a.tokens);
  if (s0 < 0 || s0 > a.tokens) { s0 = s0 < 0 ? 0 : a.tokens; q.bad = true; }
  if (s1 < s0 || s1 > a.tokens) { s1 = s1 < s0 ? s0 : a.tokens; q.bad = true; }
  if (s1 - s0 > a.max_new) { s1 = s0 + a.max_new; q.bad = true; }
  int64_t cap = a.width << a.pool.shift;
  if (cap > a.max_len) cap = a.max_len;
  if (len < 0 || len > cap) { len = len < 0 ? 0 : cap; q.bad = true; }
  q.first = s0;
  q.n = (int)(s1 - s0);
  q.len = (int)len;
  return q;
}

// Keys [lo, hi) that query i sees.
__device__ __forceinline__ int seen_hi(const AttendArgs& a, const Seq& q, int i) {
  const int at = q.len - q.n + i + 1;
  return a.causal ? (at < q.len ? at : q.len) : q.len;
}
__device__ __forceinline__ int seen_lo(const AttendArgs& a, const Seq& q, int i) {
  const int at = q.len - q.n + i + 1 - a.window;
  return a.window && at > 0 ? at : 0;
}

// Maximum and sum over the four 16-lane groups that share a query, by row
// swaps between registers (no LDS crossbar): swapping a copy of x with itself
// leaves rows 0, 0, 2, 2 in one register and 1, 1, 3, 3 in the other, then
// the halves likewise.
template <typename F>
__device__ __forceinline__ float over_groups(float x, F f) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = f(__uint_as_float(p[0]), __uint_as_float(p[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return f(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float max_groups(float x) {
  return over_groups(x, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float sum_groups(float x) {
  return over_groups(x, [](float a, float b) { return a + b; });
}

// How a cache's rows become MFMA operands.  Int8 codes and the levels of Int4
// (k) and FP4 (m, whole halves) are exact in bf16; their 1/7 and 1/6 go to the
// row's scale.  An NF4 level is not: rounded to bf16 it would be off by up to
// 2^-8, the same way in every row, which a sum over 10^5 keys does not average
// out (7 % of such an output's norm, measured); it enters as the sum of two
// bf16 values (2^-16), each with its own MFMA, or in the tile kernel as the
// product with its row's scale, rounded to fp16.
enum Operand { kOpBF16, kOpINT8, kOpLevel, kOpLevel2 };
template <int KT>
constexpr int kBitsOf = KT == kOpBF16 ? 16 : KT == kOpINT8 ? 8 : 4;

// 8 consecutive int8 codes -> 8 bf16 (exact).
__device__ __forceinline__ bf16x8 int8_to_bf16x8(uint32_t a, uint32_t b) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = (float)(int8_t)(a >> (8 * j));
    f[4 + j] = (float)(int8_t)(b >> (8 * j));
  }
  return to_bf16x8(f);
}

// Growth of a row's maximum (in powers of two) that its reference lets pass.
constexpr float kSlack = 8.0f;

// The tile kernel (attend_tile.hip): 128 rows to a tile, or 256 (quantized
// caches, heads of up to 128).
void launch_attend_tile(const AttendArgs& a, int rows, hipStream_t s);

}  // namespace qlora
