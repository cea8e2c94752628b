// Softmax cross entropy of tokens over a large vocabulary, with its gradient,
// without keeping the logits (gfx950, bf16 MFMA 32x32x16).
//
//   z_j = x . w_j,  loss = log sum_j exp(z_j) - z_t,
//   dx = g (sum_{j != t} p_j w_j  -  (1 - p_t) w_t),   p = softmax(z)
//
// x: a token's last hidden state, W [V,K] the head, which is frozen as every
// base weight of a model trained by adapters, so it gets no gradient.
//
// Two matrix products, not three: the exponentials are taken relative to a
// reference that is known before the logits are, so the first product writes
// exp(z_j) / 2^ref in bf16 at once and the second multiplies it by W; what the
// sum and its scale are is applied to the result.  The reference is the power of
// two next to the target's exponential (one dot product per token).  Tiles whose
// largest exponential is more than kLift powers above it take that one's own and
// are reported; a small kernel then brings their rows to one reference again,
// without rounding, since references are whole powers of two.  So a step
// costs 4 T K V operations where a loss and a later gradient that recomputes
// the logits would cost 6, and the target's term is left out of the
// exponentials: its weight 1 - p_t is the sum of the others, which keeps its
// digits for tokens that are nearly certain.
//
// The vocabulary is taken in pieces whose exponentials fit kPieceBytes, and
// tokens in blocks of kBlockTokens.  Tokens whose target is negative are not
// learned: the others are listed first, and only they are multiplied.
//
// Exponentials enter the second product as bf16, so dx is off by 1.7e-3 (half
// a bf16 step, root mean square) of the sum of p_j w_j beside its own rounding;
// logits, sums and the products' accumulation are fp32.
//
// Bound by matrix instructions and power: 4096 tokens of 4096 (a tenth not
// learned) over 128000 words take 6.8 ms, 1130 TFLOP/s, with the matrix units
// busy 74 % (first product) and 62 % (second, 240 tiles on 256 compute units) of
// the clocks at 1.9 GHz; a step of 64 values takes 1.55 and 1.62 us, that of the
// library's 8192^3 product 1.53.  Few tokens: memory, 262 MB of W in 43 us, 6.1 TB/s.
#include "common.hpp"
#include "device_state.hpp"
#include "timing.hpp"
#include "train.hpp"

#include <type_traits>

namespace qlora {

namespace {
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int64_t kBlockTokens = 4096;
constexpr int64_t kPieceBytes = int64_t(128) << 20;
constexpr float kLift = 58.0f;       // 2^58 leaves 2^69 of fp32's range for sums and weights
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }

// Everything a step needs, by value.
struct Loss {
  HeadLossArgs a;
  int32_t* list;    // [T] tokens that are learned, ascending
  int32_t* count;   // [1] their number
  float* tz;        // [T] the target's logit
  float* ref;       // [T] the power of two that the token's exponentials are relative to
  int32_t* lifted;  // [T] the largest reference of a lifted tile, as an ordered integer
  int32_t* flags;   // [blocks * pieces] whether any tile of the piece was lifted
  float2* stats;    // [block][nstat] (reference, sum) of each row and stretch of its columns
  uint16_t* P;      // [block][pitch] exponentials
  float* acc;       // [slabs][rows][K] sum of exponentials times W
  int64_t block;    // tokens of a block
  int64_t piece;    // columns of a piece, a multiple of 256
  int64_t pitch;    // of P
  int32_t pieces;
  int32_t nstat;
  int* status;
};

// Floats as integers in the same order (finite ones and infinities).
__device__ __forceinline__ int32_t ordered(float x) {
  const int32_t i = (int32_t)__float_as_uint(x);
  return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float from_ordered(int32_t i) { return __uint_as_float((uint32_t)(i ^ ((i >> 31) & 0x7FFFFFFF))); }
constexpr int32_t kNotLifted = INT32_MIN;

// The reference of a logit: the whole power of two next to its exponential.
__device__ __forceinline__ float ref_of(float z) { return rintf(z * kLog2e); }
// 2^d, exactly, for the whole d <= 0 by which references differ (0 where it would
// be far below every sum; no number if d is none).
__device__ __forceinline__ float pow2(float d) {
  const float x = __builtin_amdgcn_ldexpf(1.0f, (int)fmaxf(d, -300.0f));
  return d == d ? x : d;
}

// Rows of block b that are learned.
__device__ __forceinline__ int rows_of(const Loss& L, int64_t b) {
  const int64_t left = (int64_t)__builtin_amdgcn_readfirstlane(*L.count) - b * L.block;
  return left < 0 ? 0 : left < L.block ? (int)left : (int)L.block;
}
}  // namespace

// The first workgroup lists the learned tokens in ascending order and clears the
// flags; the others take four tokens each: the target's logit of a learned one,
// zeros for what the others get.
__global__ __launch_bounds__(1024) void head_begin_kernel(Loss L, int nflags) {
  __shared__ int wave_n[16];
  __shared__ float part[16];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int64_t T = L.a.T, K = L.a.K;
  if (blockIdx.x == 0) {
    for (int i = tid; i < nflags; i += 1024) L.flags[i] = 0;
    int base = 0;
    bool bad = false;
    for (int64_t t0 = 0; t0 < T; t0 += 1024) {
      const int64_t t = t0 + tid;
      const int64_t y = t < T ? L.a.targets[t] : -1;
      bad |= y >= L.a.V;
      const bool on = y >= 0 && y < L.a.V;
      const uint64_t m = __ballot(on);
      __syncthreads();
      if (lane == 0) wave_n[wave] = __popcll(m);
      __syncthreads();
      int before = base, all = 0;
      for (int w = 0; w < 16; ++w) {
        before += w < wave ? wave_n[w] : 0;
        all += wave_n[w];
      }
      if (on) L.list[before + __popcll(m & ((1ull << lane) - 1))] = (int32_t)t;
      base += all;
    }
    if (bad) atomicOr(L.status, kStatusIndex);
    if (tid == 0) *L.count = base;
    return;
  }
  const int64_t t = (int64_t)(blockIdx.x - 1) * 4 + (wave >> 2);
  const int64_t y = t < T ? L.a.targets[t] : -1;
  const bool on = y >= 0 && y < L.a.V;
  const int at = (wave & 3) * 64 + lane;
  float sum = 0.0f;
  if (on) {
    const uint16_t* x = L.a.X + t * K;
    const uint16_t* w = L.a.W + y * K;
#pragma unroll 4
    for (int64_t k = at * 8; k < K; k += 2048) {
      const u32x4 xv = *reinterpret_cast<const u32x4*>(x + k), wv = *reinterpret_cast<const u32x4*>(w + k);
#pragma unroll
      for (int q = 0; q < 4; ++q) sum += bf16_lo(xv[q]) * bf16_lo(wv[q]) + bf16_hi(xv[q]) * bf16_hi(wv[q]);
    }
  } else if (t < T) {
    if (at == 0) {
      L.a.loss[t] = 0.0f;
      L.a.lse[t] = 0.0f;
    }
    if (L.a.dX)
      for (int64_t k = at * 8; k < K; k += 2048) *reinterpret_cast<u32x4*>(L.a.dX + t * K + k) = u32x4{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off, 64);
  if (lane == 0) part[wave] = sum;
  __syncthreads();
  if (on && at == 0) {
    const float z = part[wave] + part[wave + 1] + part[wave + 2] + part[wave + 3];
    L.tz[t] = z;
    L.ref[t] = ref_of(z);
    L.lifted[t] = kNotLifted;
  }
}

// Tile shapes of the two products by the tokens of a tile.
template <int BT>
struct Shape;
template <>
struct Shape<256> {
  static constexpr int kWaves = 8, BV = 256, WV = 2, WT = 4;    // logits: vocabulary rows, waves along them and tokens
  static constexpr int BK = 256, GT = 2, GK = 4;                // gradient: columns of W, waves along tokens and them
};
template <>
struct Shape<64> {
  static constexpr int kWaves = 4, BV = 128, WV = 4, WT = 1;
  static constexpr int BK = 128, GT = 1, GK = 4;
};

// Tile n of tiles_t x others: groups of four token tiles, within one the others
// in order, so that the 32 tiles that an XCD holds at a time are four by eight
// and share their operands through its L2.
struct TileAt {
  int t, other;
};
__device__ __forceinline__ TileAt tile_at(int n, int tiles_t, int others) {
  const int g = n / (4 * others), in = n - g * 4 * others;
  const int wide = tiles_t - 4 * g < 4 ? tiles_t - 4 * g : 4;
  return TileAt{__builtin_amdgcn_readfirstlane(4 * g + in % wide), __builtin_amdgcn_readfirstlane(in / wide)};
}

// Slabs of the second product's contraction: as many as its tiles leave of the
// 256 compute units, of eight steps at least.
template <int BT>
__host__ __device__ __forceinline__ int slabs_of(int64_t rows, int64_t K, int64_t piece) {
  constexpr int BK = Shape<BT>::BK;
  const int64_t tiles = ((rows + BT - 1) / BT) * ((K + BK - 1) / BK);
  int64_t s = tiles > 0 ? 256 / tiles : 1;
  const int64_t most = piece / 512;
  if (s > most) s = most;
  if (s > 16) s = 16;
  return s < 1 ? 1 : (int)s;
}

// The main loop of both products: a workgroup's steps of 64 contracted values
// through LDS, W in three stages and the other operand, which is smaller and
// comes from the caches, in two.  A step is four substeps of A x B MFMAs; beside
// each MFMA goes a fixed share of the other work, fenced so that it stays in its
// substep (FENCED: beside its MFMA; the transposing reads of the second product
// are 2 % faster where the compiler places them): the operands of the next substep are read from LDS, and in the last substep,
// once every wave has read this step's stages for the last time (the barrier
// before it), what comes next is sent for into them.  W is on its way for two
// steps and the other operand for one, before the barrier at which a wave waits
// for all but its last loads of W.  (W in two stages: 235 for 218 us where it
// comes from memory, 512 tokens of 8192 over 32000 words.)
//   load_o(stage, step, i)  load i of LO of a step's rows (past the last: nothing)
//   load_w(stage, step, i)  the same of W, i of LW
//   read(o, w, s, i)        LDS read i of R of substep s, from stages o and w
//   mma(s, a, c)            MFMA of operands a and c
template <int A, int B, int R, int LO, int LW, bool FENCED, class LoadO, class LoadW, class Read, class Mma>
__device__ __forceinline__ void pipeline(int nk, LoadO load_o, LoadW load_w, Read read, Mma mma) {
  constexpr int N = A * B, L = LO + LW;
#pragma unroll
  for (int st = 0; st < 2; ++st) {
#pragma unroll
    for (int i = 0; i < LO; ++i) load_o(st, st, i);
#pragma unroll
    for (int i = 0; i < LW; ++i) load_w(st, st, i);
  }
#pragma unroll
  for (int i = 0; i < LW; ++i) load_w(2, 2, i);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(L + LW) : "memory");
#pragma unroll
  for (int i = 0; i < R; ++i) read(0, 0, 0, i);
  __builtin_amdgcn_sched_barrier(0);
  auto step = [&](auto phase, int kb) __attribute__((always_inline)) {
    constexpr int o = decltype(phase)::value % 2, w = decltype(phase)::value % 3;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s == 3) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LW) : "memory");
#pragma unroll
      for (int i = 0; i < N; ++i) {
        mma(s, i / B, i % B);
#pragma unroll
        for (int r = i * R / N; r < (i + 1) * R / N; ++r) read(s < 3 ? o : 1 - o, s < 3 ? w : (w + 1) % 3, (s + 1) & 3, r);
        if (s == 3)
#pragma unroll
          for (int l = i * L / N; l < (i + 1) * L / N; ++l) {
            if (l < LO) load_o(o, kb + 2, l);
            else load_w(w, kb + 3, l - LO);
          }
        if (FENCED || i == N - 1) __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  int kb = 0;
  for (; kb + 6 <= nk; kb += 6) {
    step(std::integral_constant<int, 0>{}, kb);
    step(std::integral_constant<int, 1>{}, kb + 1);
    step(std::integral_constant<int, 2>{}, kb + 2);
    step(std::integral_constant<int, 3>{}, kb + 3);
    step(std::integral_constant<int, 4>{}, kb + 4);
    step(std::integral_constant<int, 5>{}, kb + 5);
  }
  if (kb < nk) step(std::integral_constant<int, 0>{}, kb);
  if (kb + 1 < nk) step(std::integral_constant<int, 1>{}, kb + 1);
  if (kb + 2 < nk) step(std::integral_constant<int, 2>{}, kb + 2);
  if (kb + 3 < nk) step(std::integral_constant<int, 3>{}, kb + 3);
  if (kb + 4 < nk) step(std::integral_constant<int, 4>{}, kb + 4);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");  // the stages are free
}

// The stages of a kernel in LDS, each an object of its own, so that the compiler
// can tell one being filled from those being read.
struct Stages {
  unsigned char* w[3];
  unsigned char* o[2];
  // Where 64 rows of what is staged on the way out go.
  __device__ __forceinline__ unsigned char* area(int q) const {
    return q == 0 ? w[0] : q == 1 ? w[1] : q == 2 ? w[2] : o[0];
  }
};

// Sixteen bytes a lane into LDS; ONCE: marked as used once (the nt bit).
template <bool ONCE>
__device__ __forceinline__ void load_to_lds(rsrc_t r, void* lds_block, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)lds_block, 16, (int)off, 0, 0, ONCE ? 2 : 0);
}

// First product, one tile: the logits of BT tokens and BV vocabulary rows, and
// of them the sums of exponentials (one per token and wave) and, for the
// gradient, the exponentials themselves.  The contraction starts at step `first`
// and goes round.
template <int BT, int NW, int BV, int WV, int WT, bool GRAD, bool ONCE>
__device__ __forceinline__ void logits_tile(const Loss& L, int b, int pc, int rows, int r0, int64_t v0,
                                            int first, const Stages& st) {
  constexpr int A = BV / WV / 32, B = BT / WT / 32;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int l32 = lane & 31, h = lane >> 5, wv = wave % WV, wt = wave / WV;
  const int64_t K = L.a.K, V = L.a.V;
  const int64_t c0 = (int64_t)pc * L.piece, c1 = c0 + L.piece < V ? c0 + L.piece : V;
  const rsrc_t rw = make_rsrc(L.a.W + v0 * K, (V - v0) * K * 2);
  const rsrc_t rx = make_rsrc(L.a.X, L.a.T * K * 2);

  // Staging: rows of 64 values (128 bytes), eight rows to an instruction; the
  // 16-byte chunk index is XOR-ed with bits 1..3 of the row.
  constexpr int NA = BV / 8 / NW, NB = BT / 8 / NW;
  const int dr = lane >> 3, dc = lane & 7;
  uint32_t ao[NA], bo[NB];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int row = wave * (BV / NW) + 8 * i + dr;
    ao[i] = (uint32_t)(row * K * 2 + ((dc ^ ((row >> 1) & 7)) << 4));
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int row = wave * (BT / NW) + 8 * i + dr;
    const bool ok = r0 + row < rows;
    const int64_t t = ok ? L.list[b * L.block + r0 + row] : 0;
    bo[i] = ok ? (uint32_t)(t * K * 2 + ((dc ^ ((row >> 1) & 7)) << 4)) : kOffNone;
  }
  const int nk = (int)(K / 64);
  auto at = [&](int kb) __attribute__((always_inline)) {
    return kb < nk ? (uint32_t)(kb + first < nk ? kb + first : kb + first - nk) * 128 : kOffNone;
  };
  auto load_w = [&](int stage, int kb, int i) __attribute__((always_inline)) {
    load_to_lds<ONCE>(rw, st.w[stage] + (wave * (BV / NW) + 8 * i) * 128, ao[i] + at(kb));
  };
  auto load_x = [&](int stage, int kb, int i) __attribute__((always_inline)) {
    buf_load16_to_lds(rx, st.o[stage] + (wave * (BT / NW) + 8 * i) * 128, bo[i] + at(kb));
  };
  f32x16 acc[A][B];
#pragma unroll
  for (int a = 0; a < A; ++a)
#pragma unroll
    for (int c = 0; c < B; ++c)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[a][c][e] = 0.0f;
  const int sw = (l32 >> 1) & 7;
  bf16x8 oa[2][A], ob[2][B];  // operands of two substeps
  // Operand i of substep s: i < B tokens, else vocabulary rows.
  auto read = [&](int o, int w, int s, int i) __attribute__((always_inline)) {
    const int ch = ((2 * s + h) ^ sw) << 4;
    if (i < B) ob[s & 1][i] = *reinterpret_cast<const bf16x8*>(st.o[o] + (wt * (BT / WT) + 32 * i + l32) * 128 + ch);
    else oa[s & 1][i - B] = *reinterpret_cast<const bf16x8*>(st.w[w] + (wv * (BV / WV) + 32 * (i - B) + l32) * 128 + ch);
  };
  pipeline<A, B, A + B, NB, NA, true>(
      nk, load_x, load_w, read,
      [&](int s, int a, int c) __attribute__((always_inline)) { acc[a][c] = mfma32(oa[s & 1][a], ob[s & 1][c], acc[a][c]); });

  // Lane (l32, h) holds of token 32 c + l32 the logits of rows 8 (e / 4) + 4 h
  // + e % 4 of each 32-row block a.
  const int nv = (int)(c1 - v0 < BV ? c1 - v0 : BV);  // rows that exist
#pragma unroll
  for (int c = 0; c < B; ++c) {
    const int rt = r0 + wt * (BT / WT) + 32 * c + l32;
    const bool ok = rt < rows;
    const int64_t t = ok ? L.list[b * L.block + rt] : 0;
    const int64_t y = ok ? L.a.targets[t] - v0 : -1;     // the target's row of this tile, if there
    const int own = y >= 0 && y < BV ? (int)y : -1;
    const float base = ok ? L.ref[t] : 0.0f;
    // The target and rows past the last count as nothing; few tiles hold any.
    if (nv < BV || __ballot(own >= 0)) {
#pragma unroll
      for (int a = 0; a < A; ++a)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int v = wv * (BV / WV) + 32 * a + 8 * (e / 4) + 4 * h + e % 4;
          if (v >= nv || v == own) acc[a][c][e] = -INFINITY;
        }
    }
    float m = -INFINITY;
#pragma unroll
    for (int a = 0; a < A; ++a)
#pragma unroll
      for (int e = 0; e < 16; ++e) m = fmaxf(m, acc[a][c][e]);
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    const bool lift = ok && m * kLog2e - base > kLift;
    const float ref = lift ? ref_of(m) : base;
    if (GRAD && lift && h == 0) {
      atomicMax(L.lifted + t, ordered(ref));
      atomicOr(L.flags + b * L.pieces + pc, 1);
    }
    float sum = 0.0f;
#pragma unroll
    for (int a = 0; a < A; ++a)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        acc[a][c][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[a][c][e], kLog2e, -ref));
        sum += acc[a][c][e];
      }
    sum += __shfl_xor(sum, 32, 64);
    const int64_t stat = (v0 + wv * (BV / WV)) / (BV / WV);
    if (ok && h == 0 && stat < L.nstat) L.stats[(int64_t)rt * L.nstat + stat] = make_float2(ref, sum);
    if constexpr (GRAD) {
      const int tr = wt * (BT / WT) + 32 * c + l32;
      unsigned char* const row = st.area(tr / 64) + tr % 64 * (BV * 2);
#pragma unroll
      for (int a = 0; a < A; ++a)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int ch = wv * (BV / WV / 8) + 4 * a + q;
          *reinterpret_cast<uint2*>(row + ((ch ^ (l32 & (BV / 8 - 1))) << 4) + 8 * h) =
              make_uint2(pack_bf16x2(acc[a][c][4 * q], acc[a][c][4 * q + 1]),
                         pack_bf16x2(acc[a][c][4 * q + 2], acc[a][c][4 * q + 3]));
        }
    }
  }
  if constexpr (GRAD) {
    __syncthreads();
    constexpr int CH = BV / 8;  // 16-byte chunks of a row
#pragma unroll
    for (int i = 0; i < BT * CH / (64 * NW); ++i) {
      const int idx = 64 * NW * i + tid, row = idx / CH, ch = idx % CH;
      const unsigned char* p = st.area(row / 64) + row % 64 * (BV * 2) + ((ch ^ (row & 31 & (CH - 1))) << 4);
      if (r0 + row < rows)
        *reinterpret_cast<u32x4*>(L.P + (int64_t)(r0 + row) * L.pitch + (v0 - c0) + 8 * ch) =
            *reinterpret_cast<const u32x4*>(p);
    }
  }
}

// First product.  The grid is sized for whole blocks and the tiles are counted
// here; XCD x (workgroup b runs on b % 8) takes a run of them.  Where they would
// leave a last round of the 256 compute units half empty or emptier, that round
// takes tiles of half as many vocabulary rows.
template <int BT, bool GRAD, bool ONCE>
__global__ __launch_bounds__(64 * Shape<BT>::kWaves) void head_logits_kernel(Loss L, int b, int pc) {
  using S = Shape<BT>;
  constexpr int BV = S::BV;
  __shared__ __align__(1024) unsigned char w0[BV * 128], w1[BV * 128], w2[BV * 128], x0[BT * 128], x1[BT * 128];
  const Stages st{{w0, w1, w2}, {x0, x1}};
  static_assert(BT == 64 || (BT == 256 && BV <= BT), "64 rows on the way out fit a stage");
  const int rows = rows_of(L, b);
  const int64_t c0 = (int64_t)pc * L.piece, c1 = c0 + L.piece < L.a.V ? c0 + L.piece : L.a.V;
  const int tiles_t = (rows + BT - 1) / BT, tiles_v = (int)((c1 - c0 + BV - 1) / BV), tiles = tiles_t * tiles_v;
  const int rest = tiles % 256;
  const bool halves = BT == 256 && rest > 0 && rest <= 128;
  const int whole = halves ? tiles - rest : tiles, per = (whole + 7) / 8;
  const int xcd = blockIdx.x & 7, local = blockIdx.x >> 3;
  if (local < per) {
    const int n = xcd * per + local;
    if (n >= whole) return;
    const TileAt at = tile_at(n, tiles_t, tiles_v);
    // Rows of W a power of two apart lie in the same memory channels, and the tiles
    // of few tokens read theirs once, side by side: each starts at a column of its
    // own (1 token, 32000 words: 4096 values 62 -> 56 us, 8192 values 110 -> 99).
    // Larger tiles share W through the caches and stay together.
    const int first = BT == 64 ? n % (int)(L.a.K / 64) : 0;
    logits_tile<BT, S::kWaves, BV, S::WV, S::WT, GRAD, ONCE>(L, b, pc, rows, at.t * BT, c0 + (int64_t)at.other * BV, first, st);
  } else if constexpr (BT == 256) {
    const int per2 = (2 * rest + 7) / 8, n = xcd * per2 + local - per;
    if (!halves || local - per >= per2 || n >= 2 * rest) return;
    const TileAt at = tile_at(whole + n / 2, tiles_t, tiles_v);
    const int64_t v0 = c0 + (int64_t)at.other * BV + (n & 1) * (BV / 2);
    if (v0 >= c1) return;
    logits_tile<BT, 8, BV / 2, 1, 8, GRAD, ONCE>(L, b, pc, rows, at.t * BT, v0, 0, st);
  }
}

// Rows of a piece with a lifted tile: every stretch of exponentials and what
// was summed before are brought to the row's new reference (by powers of two: no
// value is rounded again).
template <int BT>
__global__ __launch_bounds__(256) void head_lift_kernel(Loss L, int b, int pc) {
  if (L.flags[b * L.pieces + pc] == 0) return;
  constexpr int kStretch = Shape<BT>::BV / Shape<BT>::WV;
  const int64_t K = L.a.K, c0 = (int64_t)pc * L.piece, c1 = c0 + L.piece < L.a.V ? c0 + L.piece : L.a.V;
  const int rows = rows_of(L, b), nslabs = slabs_of<BT>(rows, K, L.piece);
  for (int i = blockIdx.x; i < rows; i += gridDim.x) {
    const int64_t t = L.list[b * L.block + i];
    const int32_t o = L.lifted[t];
    const float old = L.ref[t], now = from_ordered(o);
    __syncthreads();  // everyone has read them
    if (o == kNotLifted || !(now > old)) continue;
    for (int64_t c = c0 + threadIdx.x * 8; c < c1; c += 256 * 8) {
      const float f = pow2(L.stats[(int64_t)i * L.nstat + c / kStretch].x - now);
      u32x4* p = reinterpret_cast<u32x4*>(L.P + (int64_t)i * L.pitch + (c - c0));
      u32x4 v = *p;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = pack_bf16x2(bf16_lo(v[q]) * f, bf16_hi(v[q]) * f);
      *p = v;
    }
    if (pc > 0) {
      const float f = pow2(old - now);
      for (int s = 0; s < nslabs; ++s)
        for (int64_t k = threadIdx.x; k < K; k += 256) L.acc[((int64_t)s * rows + i) * K + k] *= f;
    }
    if (threadIdx.x == 0) {
      L.ref[t] = now;
      L.lifted[t] = kNotLifted;
    }
  }
}

// Second product: acc[row][k] += sum over the piece of P[row][v] W[v][k].  The
// contraction is cut into slabs where the tiles alone would not fill the chip.
template <int BT, bool ONCE>
__global__ __launch_bounds__(64 * Shape<BT>::kWaves) void head_grad_kernel(Loss L, int b, int pc) {
  using S = Shape<BT>;
  constexpr int NW = S::kWaves, BK = S::BK, A = BT / S::GT / 32, B = BK / S::GK / 32;
  __shared__ __align__(1024) unsigned char w0[BK * 128], w1[BK * 128], w2[BK * 128], p0[BT * 128], p1[BT * 128];
  const Stages st{{w0, w1, w2}, {p0, p1}};
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int l32 = lane & 31, h = lane >> 5, wk = wave % S::GK, wt = wave / S::GK;
  const int rows = rows_of(L, b);
  const int tiles_t = (rows + BT - 1) / BT;
  const int64_t K = L.a.K, V = L.a.V;
  const int64_t c0 = (int64_t)pc * L.piece, c1 = c0 + L.piece < V ? c0 + L.piece : V;
  const int tiles_k = (int)((K + BK - 1) / BK);
  const int nslabs = __builtin_amdgcn_readfirstlane(slabs_of<BT>(rows, K, L.piece));
  const int whole = tiles_t * tiles_k, tiles = whole * nslabs, per = (tiles + 7) / 8;
  const int n = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || n >= tiles) return;
  const int sl = __builtin_amdgcn_readfirstlane(n / whole);
  const TileAt at = tile_at(n - sl * whole, tiles_t, tiles_k);
  const int r0 = at.t * BT;
  const int64_t k0 = (int64_t)at.other * BK;
  // This slab's steps of 64 rows of W.
  const int steps = (int)((c1 - c0 + 63) / 64), each = (steps + nslabs - 1) / nslabs;
  const int sbeg = sl * each < steps ? sl * each : steps, send = sbeg + each < steps ? sbeg + each : steps;

  const rsrc_t rp = make_rsrc(L.P + (int64_t)r0 * L.pitch, (rows - r0) * L.pitch * 2);
  constexpr int NP = BT / 8 / NW, ND = 64 * BK * 2 / 1024 / NW;  // instructions of a wave
  constexpr int WCH = BK / 8;                                     // 16-byte chunks of a row of the W tile
  uint32_t po[NP], wo[ND];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int row = wave * (BT / NW) + 8 * i + (lane >> 3);
    po[i] = (uint32_t)(row * L.pitch * 2 + (((lane & 7) ^ ((row >> 1) & 7)) << 4));
  }
#pragma unroll
  for (int i = 0; i < ND; ++i) {
    const int unit = (wave * ND + i) * 64 + lane, v = unit / WCH, ch = (unit % WCH) ^ ((v & 3) << 2);
    wo[i] = (uint32_t)((v * K + 8 * ch) * 2);
  }
  const int nk = send - sbeg;
  auto load_p = [&](int stage, int step, int i) __attribute__((always_inline)) {
    buf_load16_to_lds(rp, st.o[stage] + (wave * (BT / NW) + 8 * i) * 128,
                      po[i] + (step < nk ? (uint32_t)(sbeg + step) * 128 : kOffNone));
  };
  // W's rows from a step's first on, in a view of their own: a piece of them can
  // be larger than one.
  auto load_w = [&](int stage, int step, int i) __attribute__((always_inline)) {
    const int64_t v = c0 + (int64_t)(sbeg + step) * 64;
    const rsrc_t rw = make_rsrc(L.a.W + v * K + k0, step < nk ? ((V - v) * K - k0) * 2 : 0);
    load_to_lds<ONCE>(rw, st.w[stage] + (wave * ND + i) * 1024, wo[i]);
  };
  f32x16 acc[A][B];
#pragma unroll
  for (int a = 0; a < A; ++a)
#pragma unroll
    for (int c = 0; c < B; ++c)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[a][c][e] = 0.0f;
  const int sw = (l32 >> 1) & 7;
  // Of W's rows the lane names row (lane & 15) / 4 of four and four columns to
  // a transposing read, and gets its own column of the four rows.
  const int tr_row = 8 * h + ((lane & 15) >> 2), tr_col = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  bf16x8 oa[2][A];
  s16x4 ob[2][B][2];
  // Operand i of substep s: i < 2 B half of eight rows of W, else tokens.
  auto read = [&](int o, int w, int s, int i) __attribute__((always_inline)) {
    if (i < 2 * B) {
      const int e = i & 1, c = i >> 1;
      const int v = 16 * s + 4 * e + tr_row, col = wk * (BK / S::GK) + 32 * c + tr_col;
      ob[s & 1][c][e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)(st.w[w] + v * BK * 2 + (((col >> 3) ^ ((v & 3) << 2)) << 4) + (col & 7) * 2));
    } else {
      oa[s & 1][i - 2 * B] = *reinterpret_cast<const bf16x8*>(
          st.o[o] + (wt * (BT / S::GT) + 32 * (i - 2 * B) + l32) * 128 + (((2 * s + h) ^ sw) << 4));
    }
  };
  pipeline<A, B, A + 2 * B, NP, ND, false>(
      nk, load_p, load_w, read, [&](int s, int a, int c) __attribute__((always_inline)) {
        const uint2 lo = __builtin_bit_cast(uint2, ob[s & 1][c][0]), hi = __builtin_bit_cast(uint2, ob[s & 1][c][1]);
        acc[a][c] = mfma32(oa[s & 1][a], as_bf16x8(lo.x, lo.y, hi.x, hi.y), acc[a][c]);
      });
  // Lane (l32, h) holds column 32 c + l32 of rows 8 (e / 4) + 4 h + e % 4.
  float* const out = L.acc + (int64_t)sl * rows * K;
#pragma unroll
  for (int a = 0; a < A; ++a)
#pragma unroll
    for (int c = 0; c < B; ++c) {
      const int64_t k = k0 + wk * (BK / S::GK) + 32 * c + l32;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int row = r0 + wt * (BT / S::GT) + 32 * a + 8 * (e / 4) + 4 * h + e % 4;
        if (row < rows && k < K) {
          float* p = out + (int64_t)row * K + k;
          *p = pc > 0 ? *p + acc[a][c][e] : acc[a][c][e];
        }
      }
    }
}

// A learned token's loss, and the row of its gradient.
template <int BT>
__global__ __launch_bounds__(256) void head_finish_kernel(Loss L, int b) {
  __shared__ float red[4];
  const int i = blockIdx.x, tid = threadIdx.x, rows = rows_of(L, b);
  if (i >= rows) return;
  const int64_t K = L.a.K, t = L.list[b * L.block + i];
  const int nslabs = slabs_of<BT>(rows, K, L.piece);
  const float tz = L.tz[t];
  // The row's last reference, or a later one of a loss without gradient.
  float ref = L.ref[t];
  for (int j = tid; j < L.nstat; j += 256) ref = fmaxf(ref, L.stats[(int64_t)i * L.nstat + j].x);
#pragma unroll
  for (int off = 32; off; off >>= 1) ref = fmaxf(ref, __shfl_xor(ref, off, 64));
  if ((tid & 63) == 0) red[tid >> 6] = ref;
  __syncthreads();
  ref = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  __syncthreads();
  float sum = 0.0f;
  for (int j = tid; j < L.nstat; j += 256) {
    const float2 s = L.stats[(int64_t)i * L.nstat + j];
    sum += s.y * pow2(s.x - ref);
  }
#pragma unroll
  for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off, 64);
  if ((tid & 63) == 0) red[tid >> 6] = sum;
  __syncthreads();
  const float rest = red[0] + red[1] + red[2] + red[3];
  // The target's exponential is 2^(ref0 + part), part within half a power (held to
  // it where logits are so large that fp32 has no fractions of one).
  const float ref0 = ref_of(tz), part = __builtin_amdgcn_fmed3f(__builtin_fmaf(tz, kLog2e, -ref0), -0.5f, 0.5f);
  const float own = __builtin_amdgcn_exp2f(part) * pow2(ref0 - ref), total = rest + own;
  if (tid == 0) {
    // Each from what it is made of: beside a target far below the others, lse has
    // digits that the loss has lost.
    const bool near = ref == ref0;
    const float loss = near ? log1pf(rest / own) : __builtin_fmaf(ref - ref0, kLn2, logf(total) - part * kLn2);
    L.a.loss[t] = loss;
    L.a.lse[t] = near ? tz + loss : __builtin_fmaf(ref, kLn2, logf(total));
  }
  if (!L.a.dX) return;
  const float g = L.a.dloss ? L.a.dloss[t] : 1.0f / (float)*L.count;
  const float up = g / total, down = g * (rest / total);
  const uint16_t* w = L.a.W + L.a.targets[t] * K;
  // The row of every slab, four on their way at a time (past the last: zeros).
  const int64_t apart = (int64_t)rows * K;
  const rsrc_t sums = make_rsrc(L.acc + (int64_t)i * K, ((nslabs - 1) * apart + K) * 4);
  for (int64_t k = tid * 8; k < K; k += 2048) {
    float v[8] = {};
    for (int s0 = 0; s0 < nslabs; s0 += 4) {
      u32x4 x[4][2];
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          x[s][e] = buf_load16(sums, off_if(s0 + s < nslabs, (uint32_t)(((s0 + s) * apart + k + 4 * e) * 4)));
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += __uint_as_float(x[s][e / 4][e % 4]);
    }
    const u32x4 wv = *reinterpret_cast<const u32x4*>(w + k);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = v[2 * q] * up - down * bf16_lo(wv[q]);
      v[2 * q + 1] = v[2 * q + 1] * up - down * bf16_hi(wv[q]);
    }
    *reinterpret_cast<bf16x8*>(L.a.dX + t * K + k) = to_bf16x8(v);
  }
}

__global__ void head_zero_kernel(float* mean) {
  if (threadIdx.x == 0) *mean = 0.0f;
}

// The mean over the learned tokens (0 if there are none), summed in fp64.
__global__ __launch_bounds__(256) void head_mean_kernel(Loss L) {
  __shared__ double red[4];
  double x = 0.0;
  const int n = *L.count;
  for (int i = threadIdx.x; i < n; i += 256) x += (double)L.a.loss[L.list[i]];
#pragma unroll
  for (int off = 32; off; off >>= 1) x += __shfl_xor(x, off, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  if (threadIdx.x == 0) *L.a.mean = n > 0 ? (float)((red[0] + red[1] + red[2] + red[3]) / n) : 0.0f;
}

namespace {
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

bool small_tiles(int64_t T) { return T <= 64; }

struct Layout {
  Loss L;
  int64_t blocks;
  size_t total;
};
Layout layout(const HeadLossArgs& a, bool grad, char* ws) {
  Layout l{};
  Loss& L = l.L;
  L.a = a;
  const int64_t T = a.T, K = a.K, V = a.V;
  const bool small = small_tiles(T);
  L.block = T < kBlockTokens ? T : kBlockTokens;
  l.blocks = cdiv(T, L.block);
  int64_t piece = kPieceBytes / (2 * L.block) / 256 * 256;
  if (!grad || piece > round_up(V, 256)) piece = round_up(V, 256);
  L.piece = piece;
  L.pieces = (int32_t)cdiv(V, piece);
  L.nstat = (int32_t)cdiv(V, small ? 32 : 128);
  // Rows of P a power of two apart would meet in the same memory channels.
  L.pitch = piece + (piece % 2048 == 0 ? 128 : 0);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = ws ? ws + at : nullptr;  // (sizes alone are asked for without one)
    at += align256(bytes);
    return p;
  };
  L.list = reinterpret_cast<int32_t*>(take((size_t)T * 4));
  L.count = reinterpret_cast<int32_t*>(take(4));
  L.flags = reinterpret_cast<int32_t*>(take((size_t)l.blocks * L.pieces * 4));
  L.tz = reinterpret_cast<float*>(take((size_t)T * 4));
  L.ref = reinterpret_cast<float*>(take((size_t)T * 4));
  L.lifted = reinterpret_cast<int32_t*>(take((size_t)T * 4));
  L.stats = reinterpret_cast<float2*>(take((size_t)L.block * L.nstat * 8));
  if (grad) {
    L.P = reinterpret_cast<uint16_t*>(take((size_t)L.block * L.pitch * 2));
    // Slabs and rows are counted on the device: at most 256 tiles if there are
    // several slabs, of at most 16 times the block's rows.
    int64_t sums = small ? 256 * 64 * 128 : 256 * 256 * 256;
    if (sums > 16 * L.block * K) sums = 16 * L.block * K;
    if (sums < L.block * K) sums = L.block * K;
    L.acc = reinterpret_cast<float*>(take((size_t)sums * 4));
  }
  l.total = at;
  return l;
}

// Tiles of few tokens read W through once.  From kStreamBytes on they mark these
// loads so: 16 tokens of 4096, without and with the mark, 187 MiB of W: loss alone 47
// and 47 us, with the gradient 99 and 97; 250 MiB: 55 and 51, 121 and 115; 1000 MiB:
// 190 and 169, 422 and 378.  (125 MiB, still in the last cache from the call before:
// 38 and 44, 73 and 78.)
template <int BT, bool ONCE>
hipError_t launch_block(const Layout& l, int b, hipStream_t s) {
  using S = Shape<BT>;
  const Loss& L = l.L;
  const int tiles_t = (int)cdiv(L.block, BT);
  const bool grad = L.a.dX != nullptr;
  for (int pc = 0; pc < L.pieces; ++pc) {
    const int64_t c0 = pc * L.piece, n = L.a.V - c0 < L.piece ? L.a.V - c0 : L.piece;
    // (Half tiles of a last round: at most 256 more workgroups.)
    const unsigned grid = 8 * (unsigned)cdiv(tiles_t * cdiv(n, S::BV), 8) + (BT == 256 ? 256 : 0);
    {
      KernelTimer kt_("head_logits_kernel", s);
      if (grad) hipLaunchKernelGGL((head_logits_kernel<BT, true, ONCE>), dim3(grid), dim3(64 * S::kWaves), 0, s, L, b, pc);
      else hipLaunchKernelGGL((head_logits_kernel<BT, false, ONCE>), dim3(grid), dim3(64 * S::kWaves), 0, s, L, b, pc);
    }
    if (!grad) continue;
    {
      KernelTimer kt_("head_lift_kernel", s);
      hipLaunchKernelGGL(head_lift_kernel<BT>, dim3(256), dim3(256), 0, s, L, b, pc);
    }
    {
      KernelTimer kt_("head_grad_kernel", s);
      const unsigned g2 = 8 * (unsigned)cdiv((int64_t)tiles_t * cdiv(L.a.K, S::BK), 8);
      hipLaunchKernelGGL((head_grad_kernel<BT, ONCE>), dim3(g2 > 256 ? g2 : 256), dim3(64 * S::kWaves), 0, s, L, b, pc);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  {
    KernelTimer kt_("head_finish_kernel", s);
    hipLaunchKernelGGL(head_finish_kernel<BT>, dim3((unsigned)L.block), dim3(256), 0, s, L, b);
  }
  return hipGetLastError();
}
}  // namespace

size_t head_loss_workspace_bytes(int64_t T, int64_t K, int64_t V, bool grad) {
  if (T <= 0) return 0;
  HeadLossArgs a{};
  a.T = T;
  a.K = K;
  a.V = V;
  return layout(a, grad, nullptr).total;
}

hipError_t launch_head_loss(const HeadLossArgs& a, void* ws, hipStream_t s) {
  if (a.T == 0) {
    hipLaunchKernelGGL(head_zero_kernel, dim3(1), dim3(64), 0, s, a.mean);
    return hipGetLastError();
  }
  Layout l = layout(a, a.dX != nullptr, static_cast<char*>(ws));
  hipError_t e = hipSuccess;
  l.L.status = status_word(&e);
  if (!l.L.status) return e;
  {
    KernelTimer kt_("head_begin_kernel", s);
    hipLaunchKernelGGL(head_begin_kernel, dim3((unsigned)(1 + cdiv(a.T, 4))), dim3(1024), 0, s, l.L,
                       (int)(l.blocks * l.L.pieces));
  }
  for (int b = 0; b < l.blocks; ++b) {
    if (!small_tiles(a.T)) e = launch_block<256, false>(l, b, s);
    else if (a.V * a.K * 2 >= kStreamBytes) e = launch_block<64, true>(l, b, s);
    else e = launch_block<64, false>(l, b, s);
    if (e != hipSuccess) return e;
  }
  {
    KernelTimer kt_("head_mean_kernel", s);
    hipLaunchKernelGGL(head_mean_kernel, dim3(1), dim3(256), 0, s, l.L);
  }
  return hipGetLastError();
}

}  // namespace qlora
