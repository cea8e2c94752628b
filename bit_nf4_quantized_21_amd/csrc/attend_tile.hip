// Attention over the paged cache, many rows at a time (gfx950): prompts,
// chunks of prompts, and single tokens of large head groups.
//
// A workgroup of four or eight waves owns 32 rows per wave and walks the keys
// in tiles of 64 that it holds in LDS as bf16 (NF4: fp16), two tiles deep: the next tile's
// rows are on their way while this one is used, straight to LDS where they are
// bf16, else to registers, from where they are widened into the other half
// before the one barrier of the step.
//
// What bounds it: instructions and power.  Per tile and wave a bf16 cache takes
// 32 MFMAs (1024 clocks), 204 vector instructions of which 32 are
// exponentials, 53 LDS and 116 scalar ones; with two waves per SIMD the matrix
// units are 39 % busy and the vector units about as much, at the 1.9 to 2.0 GHz that
// the chip then holds (with zeros for data it runs 12 % faster).  52 heads of
// 4096 causal rows: 269 us, 830 TFLOP/s of what is seen (a dense product of
// 8192^3 in bf16 runs at 1258 here).  Memory is not it: all keys from one page
// take as long.  No faster: the scores of the next tile computed between this
// one's exponentials (32 registers more), operands read further ahead, 256 rows
// for bf16, heads kept together on an XCD.
//
// S^T = K Q^T by 32x32x16 MFMAs: lane (r = lane & 31, h = lane >> 5) ends up
// with the scores of query r against keys 8 (i / 4) + 4 h + i % 4 of each
// 32-key block (register i).  O^T = V^T P^T takes its 16 keys per MFMA in that
// order (element e of half h: key 4 h + e, or 8 + 4 h + e - 4), so the weights
// go from the scores' registers into the MFMA; V^T comes from the row-major
// tile by transposing LDS reads, four keys of one dim per lane.  Rows are
// swizzled in 16-byte chunks so that both reads meet every bank once.
#include "attend.hpp"

namespace qlora {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(1))) void gptr_t;
typedef __attribute__((address_space(3))) void lptr_t;

constexpr int kTileKeys = 64;

// Chunk (16 bytes) of a row at which chunk c is kept, for keys (read down the
// rows, one chunk per lane) and for values (read four rows by 64 bytes).
template <int DP>
__device__ __forceinline__ int k_chunk(int key, int c) {
  return c ^ (DP == 64 ? (key >> 1) & 7 : key & 15);
}
template <int DP>
__device__ __forceinline__ int v_chunk(int key, int c) {
  return c ^ (DP == 64 ? ((key >> 1) & 1) << 2 : (key & 3) << 2);
}

// Two fp32 as fp16, rounded to nearest even.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}
template <bool HALF>
__device__ __forceinline__ f32x16 mfma_tile(bf16x8 a, bf16x8 b, f32x16 c) {
  if constexpr (HALF) return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else return mfma32(a, b, c);
}

// Usual scales, used as they are: keys' from 2^-10 and below 2^15 (fp16 holds their
// rows), values' from 2^-5 and below 2^6 (close enough to each other for fp16
// weights).  So are 0 and what is no finite number; others are split as part *
// 2^power with 1 <= |part| < 2, but power >= -90.
__device__ __forceinline__ bool usual_key(float s) { return fabsf(s) >= 0.0009765625f && fabsf(s) < 32768.0f; }
__device__ __forceinline__ bool usual_value(float s) { return fabsf(s) >= 0.03125f && fabsf(s) < 64.0f; }
struct SplitScale {
  float part;
  int power;
};
__device__ __forceinline__ SplitScale split_scale(float s, bool usual) {
  const int e = (int)(__float_as_uint(s) >> 23 & 255u) - 127;
  const int power = usual || e == 128 || s == 0.0f ? 0 : max(e, -90);
  return {ldexpf(s, -power), power};
}

// The sequence with the n-th largest length; of more than a wave holds, the
// n-th.  (Whatever the lengths are, every sequence is some n's.)
__device__ __forceinline__ int nth_longest(const AttendArgs& a, int n) {
  if (a.batch == 1 || a.batch > 64) return n;
  const int lane = threadIdx.x & 63, len = a.lengths[min(lane, a.batch - 1)];
  int before = 0;
  for (int j = 0; j < a.batch; ++j) {
    const int other = __builtin_amdgcn_readlane(len, j);
    before += other > len || (other == len && j < lane);
  }
  return __builtin_ctzll(__ballot(lane < a.batch && before == n));
}

// LONG: a split has more keys than the list of pages covers, which is then
// renewed on the way.  (One kernel for both: 0.4 % slower over 30 calls that
// never renew it, the worst 70.1 -> 72.1 us.)
template <int OP, int DP, int WAVES, bool EXACT, bool LONG>
__global__ __launch_bounds__(64 * WAVES, DP <= 128 ? 2 : 1) void attend_tile_kernel(AttendArgs a) {
  constexpr bool CODES = OP == kOpINT8 || OP == kOpLevel;  // exact operands, scales on scores and weights
  // NF4: fp16 operands, 8 times finer than bf16 (which left outputs off by 3.3e-3
  // of the norm; now 1.75e-3, of which 1.66e-3 is their own rounding).  They are
  // kept in range by powers of two: of a query's largest element, which goes to
  // its scores, and of scales beyond the usual, of which a key's
  // goes to its scores and a value's into the exponent of its weights.  The
  // running maximum is then that of score + power, so the weights are in range
  // for the values that they multiply, row by row, and their sum takes the power
  // out again.  Weights are kept 2^UP higher, up to 2^15, so the least is 2^-35 of
  // the largest: with usual scales what 10^5 keys lose by it stays below a bf16 unit
  // of the output, whatever they hold.  (NF4 chunks and prompts take 5 to 8 % longer
  // than with bf16 operands, half of it for the choice between scales: 4 chunks of
  // 512 over 4096, 32 heads, 182 -> 193 us, 244 where the scales are not the usual
  // ones; 8192 tokens of a prompt 611 -> 652.)
  constexpr bool HALF = OP == kOpLevel2;
  constexpr float SLACK = HALF ? 4.0f : kSlack, UP = 15.0f - SLACK;
  constexpr int BITS = kBitsOf<OP>;
  constexpr bool ASYNC = OP == kOpBF16 && EXACT;         // rows go from memory to LDS as they are
  constexpr int NT = DP / 16, NB = DP / 32;
  constexpr int EL = BITS == 16 ? 8 : 16;                // elements per staged piece
  constexpr int PW = EL * BITS / 32;                     // its dwords
  constexpr int PR = DP / EL;                            // pieces of a row
  constexpr int RUN = WAVES * 64 / PR;                   // keys that the waves' pieces cover at once
  constexpr int NP = kTileKeys > RUN ? kTileKeys / RUN : 1;  // pieces per thread
  constexpr int ROWS = 32 * WAVES;
  // Each half of the two tiles is an object of its own: the compiler waits for
  // a copy into LDS before any read that might see it.
  __shared__ __align__(16) uint16_t s_k0[kTileKeys * DP], s_v0[kTileKeys * DP];
  __shared__ __align__(16) uint16_t s_k1[kTileKeys * DP], s_v1[kTileKeys * DP];
  __shared__ __align__(16) float s_sc[CODES ? 2 : 1][2][kTileKeys];
  // HALF: the powers of each key's and value's scale (a byte each), and whether
  // a wave staged one that is not 0.
  __shared__ uint32_t s_power[HALF ? 2 : 1][HALF ? kTileKeys : 1];
  __shared__ __align__(8) uint8_t s_odd[2][8];
  __shared__ __align__(16) uint8_t s_wild[2][kTileKeys];
  // Of the pages of the next kListKeys keys: their numbers, and where their rows
  // of this head start in the codes (bytes).
  __shared__ int s_page[kListKeys / 16 + 1];
  __shared__ int64_t s_at[kListKeys / 16 + 1];
  // Entries one after another: at 8 bytes each, pairs of bf16 met half of the
  // banks (the chunks below in FP4: 151 us, so 141).
  constexpr int LW = OP == kOpLevel ? 1 : 2;
  __shared__ __align__(8) uint32_t s_lut[BITS == 4 ? 256 * LW : 1];

  const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h2 = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = a.pool.heads, G = a.group;
  // The longest work goes first, so that what is left at the end is short: all
  // first splits, the longest sequence first, its last row tiles (they see the
  // most keys) first, over all heads.  Heads are fastest, so that where their
  // number is a multiple of eight each stays on one XCD, whose L2 serves its
  // keys to all of its tiles.  (Head by head, 52 heads of 4096 causal rows took
  // 20 % longer: 1.2 waves per SIMD on average, the last head's long tiles
  // alone.  Sequences as they come: 4 chunks of 300 to 512 tokens over 512 to
  // 4608, int8, 157 us, 145 in this order (132 as it is now).)
  int id = (int)blockIdx.x, next = uniform_div(id, H);
  const int h = id - next * H;
  id = next;
  next = uniform_div(id, a.tiles);
  const int tile = a.tiles - 1 - (id - next * a.tiles);
  id = next;
  const int split = uniform_div(id, a.batch), b = nth_longest(a, id - split * a.batch);
  const Seq sq = load_seq(a, b);
  if (sq.bad && tid == 0) atomicOr(a.status, kStatusIndex);
  const int rows = sq.n * G, row0 = tile * ROWS;
  if (row0 >= rows) return;
  const int i_first = uniform_div(row0, G), i_last = uniform_div(min(rows, row0 + ROWS) - 1, G);
  const int hi = seen_hi(a, sq, i_last), lo = seen_lo(a, sq, i_first);
  const int k0 = (lo & ~15) + split * a.chunk;
  if (split > 0 && k0 >= hi) return;
  const int k1 = min(hi, k0 + a.chunk);
  const int full_hi = seen_hi(a, sq, i_first), full_lo = seen_lo(a, sq, i_last);

  const int shift = a.pool.shift;
  int first_page = 0, last = 0;  // the list's first page, and its last one as counted from there
  auto list_pages = [&](int from, int to) __attribute__((always_inline)) {  // of keys [from, to)
    first_page = from >> shift;
    last = ((to - 1) >> shift) - first_page;
    for (int p = tid; p <= last; p += 64 * WAVES) {
      int page = a.pages[(int64_t)b * a.width + first_page + p];
      if (page < 0 || page >= a.pool.pages) {
        atomicOr(a.status, kStatusIndex);
        page = 0;
      }
      s_page[p] = page;
      s_at[p] = (((int64_t)page * H + h) << shift) * kv_row_bytes(a.pool.type, a.pool.dim);
    }
  };
  if (k0 < k1) list_pages(k0, LONG ? min(k1, k0 + kListKeys) : k1);
  if (BITS == 4 && tid < 256) {
    // A byte's two levels: a pair of bf16 (exact levels), or two fp32 values.
    uint32_t x = 0, y = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t v = OP == kOpLevel ? a.levels[e] & 0xFFFFu : __float_as_uint(a.values[e]);
      x = (tid & 15) == e ? v : x;
      y = (tid >> 4) == e ? v : y;
    }
    if constexpr (OP == kOpLevel) s_lut[tid] = x | (y << 16);
    else reinterpret_cast<uint2*>(s_lut)[tid] = make_uint2(x, y);
  }

  const int D = a.pool.dim;
  const float s2 = fmaxf(fabsf(a.scale2 * (CODES ? a.unit : 1.0f)), 1.2e-38f);
  const uint32_t flip = a.scale2 < 0.0f ? 0x80008000u : 0u;  // the scale's sign goes to q
  const int wrow = row0 + 32 * wave, row = wrow + r;
  const bool wave_rows = wrow < rows, ok = row < rows;
  const int qi = ok ? row / G : 0, qg = ok ? row - qi * G : 0;
  const int my_lo = seen_lo(a, sq, qi), my_hi = ok ? seen_hi(a, sq, qi) : 0;
  // Keys that some row of the wave sees.
  const int wi_first = uniform_div(min(wrow, rows - 1), G), wi_last = uniform_div(min(rows, wrow + 32) - 1, G);
  const int w_lo = seen_lo(a, sq, wi_first), w_hi = wave_rows ? seen_hi(a, sq, wi_last) : 0;
  bf16x8 q[NT];
  float row_scale = s2;  // HALF: of the row's scores
  {
    const uint16_t* p = a.q.data + (sq.first + qi) * a.q.token_stride + (int64_t)(h * G + qg) * a.q.head_stride;
    uint32_t top = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int d = t * 16 + h2 * 8;
      u32x4 w = {0, 0, 0, 0};
      if (ok && (EXACT || d < D)) w = *reinterpret_cast<const u32x4*>(p + d);
      w ^= flip;
      q[t] = as_bf16x8(w);
      if constexpr (HALF)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7FFFu, w[e] >> 16 & 0x7FFFu));
    }
    if constexpr (HALF) {
      const auto x = __builtin_amdgcn_permlane32_swap(top, top, false, false);
      const int e = (int)(max(x[0], x[1]) >> 7), power = e == 255 ? 0 : max(e, 1) - 127;
      row_scale = ldexpf(s2, power);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        u32x4 w = __builtin_bit_cast(u32x4, q[t]);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack_f16x2(ldexpf(bf16_lo(w[e]), -power), ldexpf(bf16_hi(w[e]), -power));
        q[t] = as_bf16x8(w);
      }
    }
  }
  f32x16 o[NB];
#pragma unroll
  for (int t = 0; t < NB; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[t][i] = 0.0f;
  float m = -INFINITY, l = 0.0f;
  uint32_t spoilt = 0;  // not 0: the row sees a value that is no number
  __syncthreads();

  // Piece n of a thread is chunk lane % PR of key lane / PR of a run of 64 / PR
  // keys, which lies in one page: its address is the wave's plus the lane's.
  const uint32_t row_bytes = (uint32_t)kv_row_bytes(a.pool.type, D);
  const int pc = lane % PR, wave_key = wave * (64 / PR), lane_key = lane / PR;
  const bool stages = RUN <= kTileKeys || wave_key < kTileKeys;  // eight waves may be more than the pieces
  const uint32_t lane_off = lane_key * row_bytes + pc * (PW * 4);
  uint32_t kr[ASYNC ? 1 : NP][PW], vr[ASYNC ? 1 : NP][PW];
  float scale = 0.0f;  // of a key in the first wave, of a value in the second
  float piece_ks[OP == kOpLevel2 ? NP : 1], piece_vs[OP == kOpLevel2 ? NP : 1];
  // Where the pages of the pieces of the next tile start, read a tile ahead.
  int64_t page_at[NP];
  auto read_pages = [&](int j0) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < NP; ++n)
      page_at[n] = s_at[min(((j0 + wave_key + RUN * n) >> shift) - first_page, last)];
  };
  const uint32_t in_page = (1u << shift) - 1;
  auto load = [&](uint16_t* to_k, uint16_t* to_v, int j0) __attribute__((always_inline)) {
    if (stages)
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const uint32_t row = (uint32_t)(j0 + wave_key + RUN * n) & in_page;
      const uint8_t* kp = a.pool.k + page_at[n] + row * row_bytes;
      const uint8_t* vp = a.pool.v + page_at[n] + row * row_bytes;
      if constexpr (ASYNC) {
        // Straight to LDS, lane by lane: the swizzle picks the lane's source.
        const int key = wave_key + lane_key + RUN * n;
        const uint32_t ko = lane_key * row_bytes + k_chunk<DP>(key, pc) * 16;
        const uint32_t vo = lane_key * row_bytes + v_chunk<DP>(key, pc) * 16;
        __builtin_amdgcn_global_load_lds((const gptr_t*)(kp + ko), (lptr_t*)(to_k + (wave_key + RUN * n) * DP), 16, 0, 0);
        __builtin_amdgcn_global_load_lds((const gptr_t*)(vp + vo), (lptr_t*)(to_v + (wave_key + RUN * n) * DP), 16, 0, 0);
      } else {
        // (Whole values, assigned once: assigned on two paths, the pieces were
        // kept in scratch memory.)
        typedef uint32_t piece __attribute__((ext_vector_type(PW)));
        piece x = {}, y = {};
        if (EXACT || pc * EL < D) {
          x = *reinterpret_cast<const piece*>(kp + lane_off);
          y = *reinterpret_cast<const piece*>(vp + lane_off);
        }
#pragma unroll
        for (int w = 0; w < PW; ++w) { kr[n][w] = x[w]; vr[n][w] = y[w]; }
      }
      if constexpr (OP == kOpLevel2) {
        const int page = s_page[min(((j0 + wave_key + RUN * n) >> shift) - first_page, last)];
        const int64_t at = (((int64_t)page * H + h) << shift) + row + lane_key;
        piece_ks[n] = a.pool.ks[at];
        piece_vs[n] = a.pool.vs[at];
      }
    }
    if constexpr (CODES) {
      const int j = j0 + lane, page = s_page[min((j >> shift) - first_page, last)];
      const int64_t base = (((int64_t)page * H + h) << shift) + (j & ((1 << shift) - 1));
      if (wave < 2) scale = (wave ? a.pool.vs : a.pool.ks)[base];
    }
    read_pages(j0 + kTileKeys);
  };
  // A staged piece as bf16 pairs.
  auto widen = [&](const uint32_t (&w)[PW], float sc, uint32_t (&out)[EL / 2]) __attribute__((always_inline)) {
    if constexpr (OP == kOpBF16) {
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = w[e];
    } else if constexpr (OP == kOpINT8) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        out[2 * e] = pack_bf16x2((float)(int8_t)w[e], (float)(int8_t)(w[e] >> 8));
        out[2 * e + 1] = pack_bf16x2((float)(int8_t)(w[e] >> 16), (float)(int8_t)(w[e] >> 24));
      }
    } else {
      const char* lut = reinterpret_cast<const char*>(s_lut);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const char* p = lut + lut_offset<4 * LW>(w[e / 4], e % 4);
        if constexpr (OP == kOpLevel) {
          out[e] = *reinterpret_cast<const uint32_t*>(p);
        } else {
          // Rounded as the product of the level and the scale's part: that
          // differs from row to row, so the roundings do too and average out
          // over the keys.
          const float2 f = *reinterpret_cast<const float2*>(p);
          out[e] = pack_f16x2(f.x * sc, f.y * sc);
        }
      }
    }
  };
  // A value that no row sees becomes 0; one that is not finite becomes 0 too
  // (it must not reach rows that do not see its key through 0 * inf) and its
  // key is marked: the rows that see it give NaN.  w: a piece of key `key`,
  // which PR lanes in a row hold.
  auto tame = [&](auto& w, int buf, int key, int j0) __attribute__((always_inline)) {
    const bool any = j0 + key >= lo && j0 + key < hi;
    bool bad = false;
#pragma unroll
    for (uint32_t& v : w) {
      constexpr uint32_t EXPO = HALF ? 0x7C00u : 0x7F80u;
      uint32_t x = any ? v : 0u;
      if ((x & EXPO) == EXPO) { x &= 0xFFFF0000u; bad = true; }
      if ((x & EXPO << 16) == EXPO << 16) { x &= 0xFFFFu; bad = true; }
      v = x;
    }
    const uint64_t all = __ballot(bad) >> ((lane / PR) * PR);
    if (pc == 0) s_wild[buf][key] = (all & (((uint64_t)1 << PR) - 1)) != 0;
  };
  auto on_edge = [&](int j0) __attribute__((always_inline)) { return j0 < full_lo || j0 + kTileKeys > full_hi; };
  // What is left to do for a tile once its rows are here, before the barrier.
  auto store = [&](uint16_t* to_k, uint16_t* to_v, int buf, int j0) __attribute__((always_inline)) {
    bool odd = false;
    if constexpr (!ASYNC) {
      const bool edge = on_edge(j0);
      if (stages)
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        const int key = wave_key + lane_key + RUN * n;
        uint32_t x[EL / 2], y[EL / 2];
        float ks = 1.0f, vs = 1.0f;
        if constexpr (HALF) {
          ks = piece_ks[n];
          vs = piece_vs[n];
          uint32_t powers = 0;
          const bool k_fine = usual_key(ks), v_fine = usual_value(vs);
          if (__builtin_expect(__any(!k_fine || !v_fine), 0)) {
            const SplitScale sk = split_scale(ks, k_fine), sv = split_scale(vs, v_fine);
            ks = sk.part;
            vs = sv.part;
            powers = (sk.power & 0xFF) | (sv.power & 0xFF) << 8;
            odd |= powers && j0 + key >= lo && j0 + key < hi;
          }
          if (pc == 0) s_power[buf][key] = powers;
        }
        widen(kr[n], ks, x);
        widen(vr[n], vs, y);
        if (!CODES && edge) tame(y, buf, key, j0);
#pragma unroll
        for (int c = 0; c < EL / 8; ++c) {
          const int ch = pc * (EL / 8) + c;
          *reinterpret_cast<u32x4*>(to_k + key * DP + k_chunk<DP>(key, ch) * 8) =
              u32x4{x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]};
          *reinterpret_cast<u32x4*>(to_v + key * DP + v_chunk<DP>(key, ch) * 8) =
              u32x4{y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]};
        }
      }
    }
    if constexpr (HALF) {
      odd = __any(odd);
      if (lane == 0) s_odd[buf][wave] = odd;
    }
    if constexpr (CODES) {
      if (wave == 0) {
        s_sc[buf][0][lane] = scale * s2;
      } else if (wave == 1) {
        // The codes are finite; a scale that is not is treated as such a value.
        const bool bad = (__float_as_uint(scale) & 0x7F800000u) == 0x7F800000u, any = j0 + lane >= lo && j0 + lane < hi;
        s_sc[buf][1][lane] = bad && on_edge(j0) ? 0.0f : scale;
        s_wild[buf][lane] = bad && any;
      }
    }
    __syncthreads();
    if (ASYNC && on_edge(j0)) {
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        const int key = wave_key + lane_key + RUN * n;
        u32x4* at = reinterpret_cast<u32x4*>(to_v + key * DP + pc * 8);
        uint32_t w[4] = {(*at)[0], (*at)[1], (*at)[2], (*at)[3]};
        tame(w, buf, key, j0);
        *at = u32x4{w[0], w[1], w[2], w[3]};
      }
      __syncthreads();
    }
  };

  // Where the lane's operands lie in a tile: chunk 2 t + h2 of key r (32 keys
  // further, the same), and of the four keys the lane names to a transposing
  // read, dims 32 t + its part.  The swizzles only exchange the chunks of
  // different t, so one address per t serves every key block.
  int k_at[NT], v_at[NB];
#pragma unroll
  for (int t = 0; t < NT; ++t) k_at[t] = r * DP + k_chunk<DP>(r, 2 * t + h2) * 8;
#pragma unroll
  for (int t = 0; t < NB; ++t) {
    const int key = 4 * h2 + ((lane & 15) >> 2), col = 32 * t + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    v_at[t] = key * DP + v_chunk<DP>(key, col / 8) * 8 + (col & 7);
  }

  // What the exponents are taken relative to, for a maximum m.  (From 2^23 on m - UP
  // is rounded by more than fp16 has room for; a score's own rounding is 1 there.)
  auto reference = [&](float m) __attribute__((always_inline)) {
    if constexpr (HALF) return m == -INFINITY ? 0.0f : fabsf(m) < 8388608.0f ? m - UP : m;
    return m == -INFINITY ? 0.0f : m;
  };
  auto compute = [&](const uint16_t* tk, const uint16_t* tv, int buf, int j0) __attribute__((always_inline)) {
    uint64_t odd_waves = 0;
    if constexpr (HALF) odd_waves = *reinterpret_cast<const uint64_t*>(s_odd[buf]);
    // Keys come from LDS two MFMA pairs ahead of their use.
    f32x16 s[2];
    u32x4 kf[3][2];
    auto read_k = [&](int t) __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < 2; ++c) kf[t % 3][c] = *reinterpret_cast<const u32x4*>(tk + k_at[t] + 32 * c * DP);
    };
    read_k(0);
    if (NT > 1) read_k(1);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (t + 2 < NT) read_k(t + 2);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int c = 0; c < 2; ++c) s[c] = mfma_tile<HALF>(as_bf16x8(kf[t % 3][c]), q[t], t ? s[c] : f32x16{});
    }
    // The first values are on their way while the scores become weights.
    s16x4 vf[2][2][2];  // two dim blocks at a time
    auto read_v = [&](int i) __attribute__((always_inline)) {
      const int n = i / (NB / 2), t0 = i % (NB / 2) * 2;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          vf[i % 2][t][e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(tv + v_at[t0 + t] + (16 * n + 8 * e) * DP));
    };
    read_v(0);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (CODES) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 f = *reinterpret_cast<const float4*>(&s_sc[buf][0][32 * c + 8 * i + 4 * h2]);
          s[c][4 * i] *= f.x; s[c][4 * i + 1] *= f.y; s[c][4 * i + 2] *= f.z; s[c][4 * i + 3] *= f.w;
        }
    }
    // Score * k2 + power is what the exponent is taken of.
    float k2 = CODES ? 1.0f : HALF ? row_scale : s2;
    bool odd = false;
    if constexpr (HALF) {
      odd = __builtin_amdgcn_readfirstlane((uint32_t)odd_waves | (WAVES > 4 ? (uint32_t)(odd_waves >> 32) : 0u)) != 0;
      if (__builtin_expect(odd, 0)) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int power = (int)s_power[buf][32 * c + 8 * (i / 4) + i % 4 + 4 * h2];
            s[c][i] = __builtin_fmaf(ldexpf(s[c][i], (int8_t)power), k2, (float)(int8_t)(power >> 8));
          }
        k2 = 1.0f;
      }
    }
    if (on_edge(j0)) {
      // Bounds of the keys that the lane's row sees, against the register's own
      // place 32 c + 8 (i / 4) + i % 4.
      const int from = my_lo - j0 - 4 * h2, to = my_hi - j0 - 4 * h2;
      // Values that are no numbers spoil the outputs of the rows that see them;
      // the scores, and so the log-sum, stay.  (Rare: a loop, which needs no
      // registers beside the scores.)
      if (__any(reinterpret_cast<const uint32_t*>(s_wild[buf])[lane & 15] != 0))
#pragma unroll 1
        for (int key = 0; key < kTileKeys; ++key)
          if (j0 + key >= my_lo && j0 + key < my_hi) spoilt |= s_wild[buf][key];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int at = 32 * c + 8 * (i / 4) + i % 4;
          if (at < from || at >= to) s[c][i] = -INFINITY;
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s[0][i]);
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, s[1][i]);
    {
      const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
      top = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1])) * k2;
    }
    if (__any(top > m + SLACK)) {
      top = fmaxf(top, m);
      const float f = top == -INFINITY ? 1.0f : m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(reference(m) - reference(top));
      l *= f;
#pragma unroll
      for (int t = 0; t < NB; ++t) o[t] *= f;
      m = top;
    }
    const float ref = reference(m);
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[c][i] = __builtin_amdgcn_exp2f(CODES ? s[c][i] - ref : __builtin_fmaf(s[c][i], k2, -ref));
        sum += s[c][i];
      }
    if (HALF && __builtin_expect(odd, 0)) {
      sum = 0.0f;
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          sum += ldexpf(s[c][i], -(int8_t)(s_power[buf][32 * c + 8 * (i / 4) + i % 4 + 4 * h2] >> 8));
    }
    l += sum;
    if constexpr (CODES) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 f = *reinterpret_cast<const float4*>(&s_sc[buf][1][32 * c + 8 * i + 4 * h2]);
          s[c][4 * i] *= f.x; s[c][4 * i + 1] *= f.y; s[c][4 * i + 2] *= f.z; s[c][4 * i + 3] *= f.w;
        }
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      // The weights enter the second product as one bf16 (or fp16) value each,
      // after the row's scale where the rows are codes; their sum stays fp32.
      // As two bf16 values, like in the kernel for few rows, outputs are as good
      // as their own rounding (1.6e-3 of the norm, against 2.0e-3 to 2.4e-3 this
      // way), but the second product's MFMAs double: 52 heads of 4096 rows 276 ->
      // 357 us, 4 chunks of 512 over 4096, 32 heads, int8 190 -> 231.
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = s[n / 2][8 * (n % 2) + e];
      const bf16x8 pb = HALF ? as_bf16x8(pack_f16x2(p[0], p[1]), pack_f16x2(p[2], p[3]), pack_f16x2(p[4], p[5]), pack_f16x2(p[6], p[7]))
                             : to_bf16x8(p);
#pragma unroll
      for (int t = 0; t < NB; ++t) {
        const int i = (n * NB + t) / 2;
        if (t % 2 == 0) {
          if (i + 1 < 2 * NB) read_v(i + 1);
          __builtin_amdgcn_sched_barrier(0);
        }
        const uint2 x = __builtin_bit_cast(uint2, vf[i % 2][t % 2][0]), y = __builtin_bit_cast(uint2, vf[i % 2][t % 2][1]);
        o[t] = mfma_tile<HALF>(as_bf16x8(x.x, x.y, y.x, y.y), pb, o[t]);
      }
    }
  };

  for (int from = k0; from < k1;) {  // as many keys as the list covers
    const int to = LONG ? min(k1, from + kListKeys) : k1;
    read_pages(from);
    load(s_k0, s_v0, from);
    store(s_k0, s_v0, 0, from);
    auto step = [&](uint16_t* k, uint16_t* v, uint16_t* next_k, uint16_t* next_v, int buf, int j0) __attribute__((always_inline)) {
      const bool more = j0 + kTileKeys < to;
      if (more) load(next_k, next_v, j0 + kTileKeys);
      if (j0 < w_hi && j0 + kTileKeys > w_lo) compute(k, v, buf, j0);
      if (more) store(next_k, next_v, buf ^ 1, j0 + kTileKeys);
      return more;
    };
    for (int j0 = from;; j0 += 2 * kTileKeys) {
      if (!step(s_k0, s_v0, s_k1, s_v1, 0, j0)) break;
      if (!step(s_k1, s_v1, s_k0, s_v0, 1, j0 + kTileKeys)) break;
    }
    from = to;
    if (!LONG || from >= k1) break;
    // No wave has read the list since the last barrier; past the next one all
    // are done with the tiles.
    list_pages(from, min(k1, from + kListKeys));
    __syncthreads();
  }

  {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    l = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  if (spoilt)
#pragma unroll
    for (int t = 0; t < NB; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[t][i] = __uint_as_float(0x7FC00000u);
  if (!ok) return;
  if (HALF && m != -INFINITY) m = reference(m);  // what the sums are relative to
  const int Hq = H * G;
  const int64_t at = (sq.first + qi) * Hq + h * G + qg;
  if (hi - (lo & ~15) > a.chunk) {  // the other splits' part is to come
    const int64_t to = (int64_t)split * a.tokens * Hq + at;
    if (h2 == 0) {
      a.part_ml[2 * to] = m;
      a.part_ml[2 * to + 1] = l;
    }
#pragma unroll
    for (int t = 0; t < NB; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = 32 * t + 8 * i + 4 * h2;
        if (EXACT || d < D)
          *reinterpret_cast<float4*>(a.part_o + to * D + d) =
              make_float4(o[t][4 * i], o[t][4 * i + 1], o[t][4 * i + 2], o[t][4 * i + 3]);
      }
    return;
  }
  const float inv = l == 0.0f ? 0.0f : (CODES ? a.unit : 1.0f) / l;
  if (h2 == 0 && a.lse) a.lse[at] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
#pragma unroll
  for (int t = 0; t < NB; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = 32 * t + 8 * i + 4 * h2;
      if (EXACT || d < D)
        *reinterpret_cast<uint2*>(a.out + at * D + d) =
            make_uint2(pack_bf16x2(o[t][4 * i] * inv, o[t][4 * i + 1] * inv),
                       pack_bf16x2(o[t][4 * i + 2] * inv, o[t][4 * i + 3] * inv));
    }
}

template <int OP, int DP, int WAVES, bool LONG>
void tile_long(const AttendArgs& a, dim3 grid, hipStream_t s) {
  if (a.pool.dim == DP) hipLaunchKernelGGL((attend_tile_kernel<OP, DP, WAVES, true, LONG>), grid, dim3(64 * WAVES), 0, s, a);
  else hipLaunchKernelGGL((attend_tile_kernel<OP, DP, WAVES, false, LONG>), grid, dim3(64 * WAVES), 0, s, a);
}
template <int OP, int DP, int WAVES>
void tile_dim(const AttendArgs& a, dim3 grid, hipStream_t s) {
  if (a.chunk > kListKeys) tile_long<OP, DP, WAVES, true>(a, grid, s);
  else tile_long<OP, DP, WAVES, false>(a, grid, s);
}
template <int OP>
void tile_op(const AttendArgs& a, int rows, dim3 grid, hipStream_t s) {
  if constexpr (OP != kOpBF16) {
    if (rows == 256) {
      if (a.pool.dim <= 64) tile_dim<OP, 64, 8>(a, grid, s);
      else tile_dim<OP, 128, 8>(a, grid, s);
      return;
    }
  }
  if (a.pool.dim <= 64) tile_dim<OP, 64, 4>(a, grid, s);
  else if (a.pool.dim <= 128) tile_dim<OP, 128, 4>(a, grid, s);
  else tile_dim<OP, 256, 4>(a, grid, s);
}

}  // namespace

void launch_attend_tile(const AttendArgs& a, int rows, hipStream_t s) {
  const int64_t total = (int64_t)a.batch * a.pool.heads * a.tiles * a.splits;
  const dim3 grid((unsigned)total);
  if (a.pool.type == kKVBF16) tile_op<kOpBF16>(a, rows, grid, s);
  else if (a.pool.type == kKVINT8) tile_op<kOpINT8>(a, rows, grid, s);
  else if (a.pool.type == kKVNF4) tile_op<kOpLevel2>(a, rows, grid, s);
  else tile_op<kOpLevel>(a, rows, grid, s);
}

}  // namespace qlora
