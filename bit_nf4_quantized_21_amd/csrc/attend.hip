// Attention of new tokens over the paged key/value cache (gfx950).
//
// Query i of a sequence with n new tokens and `length` stored ones (the new
// ones among them) stands at position length - n + i and sees the keys j with
// j < length, j <= position (causal) and j > position - window (window > 0):
//     s_j = scale q.k_j,   out = sum_j exp(s_j) v_j / sum_j exp(s_j),
//     lse = log sum_j exp(s_j);   a query that sees nothing gives 0 and -inf.
// One pass over the keys with a running maximum and sum per query, in fp32 and
// base 2.  The queries of a group of heads share their key/value head, so a
// tile's rows are (token, head of the group) pairs of one key/value head.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "attend.hpp"
#include "timing.hpp"

namespace qlora {

namespace {

// The levels of the two codes in byte q of x, from the LDS table at address 0
// (`lut`): an entry per byte, a bf16 pair, or for kOpLevel2 that and the pair
// of what it misses.  (A table of 16 single codes, whose reads never meet in a
// bank, needs twice the reads and four more instructions a pair: 131071 NF4
// keys 54.7 us, 48 with it for the keys alone, 43 this way.)
template <int KT>
__device__ __forceinline__ uint2 level_pair(const uint32_t* lut, uint32_t x, int q) {
  const char* p = reinterpret_cast<const char*>(lut);
  if constexpr (KT == kOpLevel2) return *reinterpret_cast<const uint2*>(p + lut_offset<8>(x, q));
  return make_uint2(*reinterpret_cast<const uint32_t*>(p + lut_offset<4>(x, q)), 0u);
}

// Four bytes' levels as MFMA operands: the levels, or levels and rests.
template <int KT, int N>
__device__ __forceinline__ void pack_levels(const uint2 (&w)[4], bf16x8 (&out)[N]) {
  if constexpr (KT == kOpLevel2) {
    out[0] = as_bf16x8(w[0].x, w[0].y, w[1].x, w[1].y);
    out[N - 1] = as_bf16x8(w[2].x, w[2].y, w[3].x, w[3].y);
  } else {
    out[0] = as_bf16x8(w[0].x, w[1].x, w[2].x, w[3].x);
  }
}

// ---------------------------------------------------------------------------
// Streaming kernel: 16 * NQ rows of one sequence and key/value head against
// one split of its keys.  Each of the WAVES waves takes every WAVES-th step of
// 32 keys straight from memory into MFMA operands, with its own running maximum
// and sum; the waves meet once, in LDS, at the end.  What bounds it: memory
// where the cache holds 8 or 16 bits (64 sequences of up to 8192 tokens, int8:
// 650 MB in 144 us, 4.5 TB/s; 131071 keys of 8 heads 5.2 TB/s, bf16 5.8), the
// lookups and the instructions of a step where it holds 4 (131071 NF4 keys:
// 143 MB in 42 us, 3.4 TB/s; Int4 37 us; int8 39 us when the rows come from the
// caches; the join of 5 us is not in these).
//
// S^T = K Q^T by 16x16x32 MFMAs: lane (r = lane & 15, g = lane >> 4) loads the
// contiguous dims [g DP/4, (g + 1) DP/4) of key r (of each 16-key block) and
// of query r, so a row is read by four lanes and the dims' order inside the
// contraction is the same on both sides.  The scores of query r and keys
// 4g..4g+3 of each block land on lane (r, g).  O^T = V^T P^T takes its keys in
// that order: element e of lane group g is key 4g + e of block 0 (e < 4) or
// key 4g + e - 4 of block 1, so the weights go from registers to the MFMA as
// they are, and lane (r, g) loads dims [r DP/16, (r + 1) DP/16) of those 8
// keys; MFMA m of the DP/16 takes dim m of each.
// ---------------------------------------------------------------------------
template <int KT, int DP, int NQ, int WAVES, bool EXACT>
__global__ __launch_bounds__(64 * WAVES) void attend_stream_kernel(AttendArgs a) {
  constexpr bool FOUR = KT == kOpLevel || KT == kOpLevel2;
  constexpr int BITS = kBitsOf<KT>;
  constexpr int NT = DP / 32;               // QK steps
  constexpr int NM = DP / 16;               // PV MFMAs
  constexpr int KW = DP / 4 * BITS / 32;    // dwords of a key's quarter row
  constexpr int VB = DP / 16 * BITS / 8;    // bytes of a value's sixteenth row
  constexpr int VW = VB < 4 ? 1 : VB / 4;
  constexpr int OS = DP + 4;                // padded LDS row of the outputs
  constexpr int STEP = 32 * WAVES;          // keys of a step of all waves
  constexpr int TQ = 4 * WAVES;             // threads of a row at the end
  constexpr int DT = DP / TQ;               // and their dims
  // One LDS object with the table of levels first: at address 0 a byte's
  // offset is its address.
  struct __align__(16) Shared {
    uint32_t lut[KT == kOpLevel2 ? 512 : KT == kOpLevel ? 256 : 4];
    float o[WAVES * 16 * OS];
    float m[WAVES][16 * NQ], l[WAVES][16 * NQ];
    int page[kMaxChunk / 16 + 1];
  };
  __shared__ Shared sh;
  auto& s_lut = sh.lut;
  auto& s_o = sh.o;
  auto& s_m = sh.m;
  auto& s_l = sh.l;
  auto& s_page = sh.page;

  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Heads fastest: consecutive workgroups go to the eight XCDs in turn, so each
  // gets its share of every sequence, and the splits that only long sequences
  // have come last.
  const int H = a.pool.heads;
  int id = (int)blockIdx.x, next = uniform_div(id, H);
  const int h = id - next * H;
  id = next;
  next = uniform_div(id, a.batch);
  const int b = id - next * a.batch, split = uniform_div(next, a.tiles), tile = next - split * a.tiles;
  // Without a window a split's first page is known before the lengths are: its
  // pages are read with them (entries of the table past a sequence's own are
  // read but not used).
  const int shift = a.pool.shift, ahead = ((split * a.chunk) >> shift) + tid;
  int early = 0;
  if (!a.window && ahead < a.width) early = a.pages[(int64_t)b * a.width + ahead];
  const Seq sq = load_seq(a, b);
  if (sq.bad && tid == 0) atomicOr(a.status, kStatusIndex);
  const int G = a.group, rows = sq.n * G, row0 = tile * 16 * NQ;
  if (row0 >= rows) return;
  const int i_first = uniform_div(row0, G), i_last = uniform_div(min(rows, row0 + 16 * NQ) - 1, G);
  const int hi = seen_hi(a, sq, i_last), lo = seen_lo(a, sq, i_first);
  const int k0 = (lo & ~15) + split * a.chunk;
  if (split > 0 && k0 >= hi) return;
  const int k1 = min(hi, k0 + a.chunk);
  const bool several = hi - (lo & ~15) > a.chunk;  // splits, that the join puts together
  // Steps inside [full_lo, full_hi) are seen by every row.
  const int full_hi = seen_hi(a, sq, i_first), full_lo = seen_lo(a, sq, i_last);

  const int first_page = k0 >> shift, last = ((k1 - 1) >> shift) - first_page;
  for (int p = tid; k0 < k1 && p <= last; p += 64 * WAVES) {
    int page = !a.window && p == tid ? early : a.pages[(int64_t)b * a.width + first_page + p];
    if (page < 0 || page >= a.pool.pages) {
      atomicOr(a.status, kStatusIndex);
      page = 0;
    }
    s_page[p] = page;
  }
  if (FOUR && tid < 256) {
    uint32_t x = a.levels[0], y = a.levels[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) {
      x = (tid & 15) == e ? a.levels[e] : x;
      y = (tid >> 4) == e ? a.levels[e] : y;
    }
    const uint32_t pair = (x & 0xFFFFu) | (y << 16), rest = (x >> 16) | (y & 0xFFFF0000u);
    if constexpr (KT == kOpLevel2) reinterpret_cast<uint2*>(s_lut)[tid] = make_uint2(pair, rest);
    else s_lut[tid] = pair;
  }

  const int D = a.pool.dim;
  // Queries: row m of the tile is token m / G, head h * G + m % G.
  // (With two bf16 values per level a lane's 8 operand elements are two pairs
  // of codes: (level, level, rest, rest) twice, against each pair of q twice.)
  constexpr int QW = KT == kOpLevel2 ? 2 : 1;
  bf16x8 q[NQ][NT][QW];
  int my_lo[NQ], my_hi[NQ];
#pragma unroll
  for (int x = 0; x < NQ; ++x) {
    const int row = row0 + 16 * x + r;
    const bool ok = row < rows;
    const int i = ok ? row / G : 0, gh = ok ? row - i * G : 0;
    my_lo[x] = seen_lo(a, sq, i);
    my_hi[x] = ok ? seen_hi(a, sq, i) : 0;
    const uint16_t* p = a.q.data + (sq.first + i) * a.q.token_stride + (int64_t)(h * G + gh) * a.q.head_stride;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int d = g * (DP / 4) + t * 8;
      u32x4 w = {0, 0, 0, 0};
      if (ok && (EXACT || d < D)) w = *reinterpret_cast<const u32x4*>(p + d);
      if constexpr (KT == kOpLevel2) {
        q[x][t][0] = as_bf16x8(w[0], w[0], w[1], w[1]);
        q[x][t][QW - 1] = as_bf16x8(w[2], w[2], w[3], w[3]);
      } else {
        q[x][t][0] = as_bf16x8(w);
      }
    }
  }
  __syncthreads();

  f32x4 o[NQ][NM];
  float m[NQ], l[NQ];
#pragma unroll
  for (int x = 0; x < NQ; ++x) {
    m[x] = -INFINITY;
    l[x] = 0.0f;
#pragma unroll
    for (int t = 0; t < NM; ++t) o[x][t] = f32x4{0, 0, 0, 0};
  }

  const int64_t row_bytes = kv_row_bytes(a.pool.type, D);
  const uint32_t k_off = r * (uint32_t)row_bytes + g * (DP / 4) * BITS / 8;
  const uint32_t v_off = 4 * g * (uint32_t)row_bytes + r * VB;
  const float s2 = a.scale2 * a.unit;

  // A step's rows as they are stored.
  struct Stage {
    uint32_t k[2][KW], v[8][VW];
    float4 ks[2], vs[2];
  } st;
  // First row of a 16-key block (blocks lie within a page).
  auto block = [&](int j) -> int64_t {
    // The second block's page may lie past the list: its keys are not seen.
    const int page = __builtin_amdgcn_readfirstlane(s_page[min((j >> shift) - first_page, last)]);
    return (((int64_t)page * H + h) << shift) + (j & ((1 << shift) - 1));
  };
  auto load_k = [&](int j0) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int64_t base = block(j0 + 16 * c);
      const uint8_t* kp = a.pool.k + base * row_bytes + k_off;
      if constexpr (EXACT) {
        if constexpr (KW % 4 == 0) {
#pragma unroll
          for (int w = 0; w < KW; w += 4) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(kp + 4 * w);
            st.k[c][w] = v[0]; st.k[c][w + 1] = v[1]; st.k[c][w + 2] = v[2]; st.k[c][w + 3] = v[3];
          }
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(kp);
          st.k[c][0] = v.x; st.k[c][1] = v.y;
        }
      } else {
        constexpr int SW = KW / NT;  // dwords of 8 elements
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const bool in = g * (DP / 4) + t * 8 < D;
#pragma unroll
          for (int w = 0; w < SW; ++w) st.k[c][t * SW + w] = in ? reinterpret_cast<const uint32_t*>(kp)[t * SW + w] : 0u;
        }
      }
      if constexpr (KT != kOpBF16) st.ks[c] = reinterpret_cast<const float4*>(a.pool.ks + base)[g];
    }
  };
  auto load_v = [&](int j0) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int64_t base = block(j0 + 16 * c);
      const uint8_t* vb = a.pool.v + base * row_bytes;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint8_t* vp = vb + v_off + e * (uint32_t)row_bytes;
        uint32_t(&w)[VW] = st.v[4 * c + e];
        if (EXACT || r * (DP / 16) < D) {
          if constexpr (VB >= 16) {
#pragma unroll
            for (int x = 0; x < VW; x += 4) {
              const u32x4 v = *reinterpret_cast<const u32x4*>(vp + 4 * x);
              w[x] = v[0]; w[x + 1] = v[1]; w[x + 2] = v[2]; w[x + 3] = v[3];
            }
          } else if constexpr (VB == 8) {
            const uint2 v = *reinterpret_cast<const uint2*>(vp);
            w[0] = v.x; w[1] = v.y;
          } else if constexpr (VB == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(vp);
          } else {
            w[0] = *reinterpret_cast<const uint16_t*>(vp);
          }
        } else {
#pragma unroll
          for (int x = 0; x < VW; ++x) w[x] = 0;
        }
      }
      if constexpr (KT != kOpBF16) st.vs[c] = reinterpret_cast<const float4*>(a.pool.vs + base)[g];
    }
  };

  // Levels of dims t .. t + TG - 1 of the lane's 8 values: the codes of two
  // keys, side by side in a byte, name both levels.
  constexpr int TG = 4;
  uint2 vl[FOUR ? 2 : 1][TG][4];
  auto look_up = [&](int t0) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t va = st.v[2 * c][t0 / 8], vb = st.v[2 * c + 1][t0 / 8];
      const uint32_t even = (va & 0x0F0F0F0Fu) | ((vb << 4) & 0xF0F0F0F0u);
      const uint32_t odd = ((va >> 4) & 0x0F0F0F0Fu) | (vb & 0xF0F0F0F0u);
#pragma unroll
      for (int t = 0; t < TG; ++t)
        vl[t0 / TG % 2][t][c] = level_pair<KT>(s_lut, t & 1 ? odd : even, (t0 + t) % 8 / 2);
    }
  };

  // One step; the next one's keys load once this one's are used up, and its
  // values likewise: loads are always in flight, in the same registers.
  auto compute = [&](int j0, int next) {
    f32x4 s[NQ][2];
#pragma unroll
    for (int x = 0; x < NQ; ++x) s[x][0] = s[x][1] = f32x4{0, 0, 0, 0};
    // 4 bits: the lookups of a group go out before the group before it is used
    // (the fences keep the compiler from pairing each with its use, which would
    // wait for LDS at every one).
    constexpr int KG = NT < 4 ? NT : 4;
    uint2 kl[FOUR ? 2 : 1][KG][4];
    auto look_up_k = [&](int n) {
#pragma unroll
      for (int t = 0; t < KG; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          kl[n % 2][t][e] = level_pair<KT>(s_lut, st.k[(n * KG + t) / NT][(n * KG + t) % NT], e);
    };
    if constexpr (FOUR) look_up_k(0);
#pragma unroll
    for (int n = 0; n < 2 * NT; ++n) {
      const int c = n / NT, t = n % NT;
      bf16x8 ka[QW];
      if constexpr (KT == kOpBF16) {
        ka[0] = as_bf16x8(st.k[c][4 * t], st.k[c][4 * t + 1], st.k[c][4 * t + 2], st.k[c][4 * t + 3]);
      } else if constexpr (KT == kOpINT8) {
        ka[0] = int8_to_bf16x8(st.k[c][2 * t], st.k[c][2 * t + 1]);
      } else {
        if (n % KG == 0) {
          if (n + KG < 2 * NT) look_up_k(n / KG + 1);
          __builtin_amdgcn_sched_barrier(0);
        }
        pack_levels<KT>(kl[n / KG % 2][n % KG], ka);
      }
#pragma unroll
      for (int w = 0; w < QW; ++w)
#pragma unroll
        for (int x = 0; x < NQ; ++x) s[x][c] = mfma16(ka[w], q[x][t][w], s[x][c]);
    }

    if constexpr (KT != kOpBF16) {
#pragma unroll
      for (int x = 0; x < NQ; ++x)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[x][e / 4][e % 4] *= reinterpret_cast<const float*>(&st.ks[e / 4])[e % 4];
    }
    load_k(next);

    const bool edge = j0 < full_lo || j0 + 32 > full_hi;
    // Keys of the edge: those that no row of the tile sees hold anything (the
    // tail of a page, a page that was given back), so their values become 0;
    // a bf16 value that is not finite must not reach rows that do not see its
    // key through 0 * inf, so it becomes 0 too and the rows that do see it get
    // a NaN weight instead.
    uint32_t wild = 0;
    if (KT == kOpBF16 && edge) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = j0 + 16 * (e / 4) + 4 * g + e % 4;
        const bool any = j >= lo && j < hi;
        bool bad = false;
#pragma unroll
        for (int x = 0; x < VW; ++x) {
          uint32_t w = any ? st.v[e][x] : 0u;
          if ((w & 0x7F80u) == 0x7F80u) { w &= 0xFFFF0000u; bad = true; }
          if ((w & 0x7F800000u) == 0x7F800000u) { w &= 0xFFFFu; bad = true; }
          st.v[e][x] = w;
        }
        wild |= ((__ballot(bad) >> (16 * g)) & 0xFFFFu) != 0 ? 1u << e : 0u;
      }
    }

    if constexpr (FOUR) {
      look_up(0);
      __builtin_amdgcn_sched_barrier(0);
    }
    bf16x8 pb[NQ][2][QW];
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = s[x][e / 4][e % 4] * s2;
      uint32_t hidden = 0;
      if (edge) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int at = 16 * (e / 4) + e % 4;
          if (at < my_lo[x] - j0 - 4 * g || at >= my_hi[x] - j0 - 4 * g) {
            hidden |= 1u << e;
            p[e] = -INFINITY;
          }
        }
      }
      // The reference of the exponents follows the maximum only when it has
      // grown by 2^kSlack: weights stay below 2^kSlack and nothing is rescaled
      // in nearly every step.
      float top = fmaxf(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])), fmaxf(fmaxf(p[4], p[5]), fmaxf(p[6], p[7])));
      top = max_groups(top);
      if (__any(top > m[x] + kSlack)) {
        top = fmaxf(top, m[x]);
        const float f = top == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[x] - top);
        l[x] *= f;
#pragma unroll
        for (int t = 0; t < NM; ++t) o[x][t] *= f;
        m[x] = top;
      }
      const float ref = m[x] == -INFINITY ? 0.0f : m[x];
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = __builtin_amdgcn_exp2f(p[e] - ref);
      l[x] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
      if constexpr (KT != kOpBF16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] *= reinterpret_cast<const float*>(&st.vs[e / 4])[e % 4];
        if (edge) {
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e] = (hidden >> e) & 1u ? 0.0f : p[e];  // also where the scale is no number
        }
      } else if (edge) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((wild & ~hidden) >> e & 1u) p[e] = __uint_as_float(0x7FC00000u);
      }
      // The weights enter the second product as two bf16 values, their sum off
      // by 2^-16: one alone (2^-8) would show beside the output's own rounding,
      // and the matrix units have time while the rows stream.
      uint32_t w[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[0][e] = pack_bf16x2(p[2 * e], p[2 * e + 1]);
        w[1][e] = pack_bf16x2(p[2 * e] - bf16_lo(w[0][e]), p[2 * e + 1] - bf16_hi(w[0][e]));
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if constexpr (KT == kOpLevel2) {
          pb[x][n][0] = as_bf16x8(w[n][0], w[n][0], w[n][1], w[n][1]);
          pb[x][n][QW - 1] = as_bf16x8(w[n][2], w[n][2], w[n][3], w[n][3]);
        } else {
          pb[x][n][0] = as_bf16x8(w[n][0], w[n][1], w[n][2], w[n][3]);
        }
      }
    }

    // Values of dim t for the lane's 8 keys, two keys to a dword; for 4 bits
    // the lookups of a group of dims go out while the last group is used.
#pragma unroll
    for (int t = 0; t < NM; ++t) {
      bf16x8 vt[QW];
      if constexpr (FOUR) {
        if (t % TG == 0) {
          if (t + TG < NM) look_up(t + TG);
          __builtin_amdgcn_sched_barrier(0);
        }
        pack_levels<KT>(vl[t / TG % 2][t % TG], vt);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t(&va)[VW] = st.v[2 * c];
          const uint32_t(&vb)[VW] = st.v[2 * c + 1];
          if constexpr (KT == kOpBF16)
            w[c] = __builtin_amdgcn_perm(vb[t / 2], va[t / 2], t & 1 ? 0x07060302u : 0x05040100u);
          else
            w[c] = pack_bf16x2((float)(int8_t)(va[t / 4] >> (8 * (t % 4))), (float)(int8_t)(vb[t / 4] >> (8 * (t % 4))));
        }
        vt[0] = as_bf16x8(w[0], w[1], w[2], w[3]);
      }
#pragma unroll
      for (int n = 0; n < QW; ++n)
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
          o[x][t] = mfma16(vt[n], pb[x][1][n], o[x][t]);
          o[x][t] = mfma16(vt[n], pb[x][0][n], o[x][t]);
        }
    }
    load_v(next);
  };

  int j = k0 + 32 * wave;
  if (j < k1) {
    const int end = j + (k1 - 1 - j) / STEP * STEP;  // this wave's last step
    load_k(j);
    load_v(j);
    // Past the last step the rows loaded are its own again: a load that may
    // not happen would make the wait for the ones before it a wait for all.
    for (; j < k1; j += STEP) compute(j, min(j + STEP, end));
  }

  // The waves' sums meet.  Lane (r, g) holds, of query r, the dims
  // g DP/4 + i NM + t (register i of MFMA t).
#pragma unroll
  for (int x = 0; x < NQ; ++x) {
    l[x] = sum_groups(l[x]);
    if (g == 0) {
      s_m[wave][16 * x + r] = m[x];
      s_l[wave][16 * x + r] = l[x];
    }
  }
  __syncthreads();
  const int Hq = H * G;
#pragma unroll
  for (int x = 0; x < NQ; ++x) {
    {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) top = fmaxf(top, s_m[w][16 * x + r]);
      const float f = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[x] - top);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < NM; t += 4)
          *reinterpret_cast<float4*>(s_o + (wave * 16 + r) * OS + g * (DP / 4) + i * NM + t) =
              make_float4(o[x][t][i] * f, o[x][t + 1][i] * f, o[x][t + 2][i] * f, o[x][t + 3][i] * f);
    }
    __syncthreads();
    const int qr = tid / TQ, part = tid % TQ, row = row0 + 16 * x + qr;
    if (row < rows) {
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) top = fmaxf(top, s_m[w][16 * x + qr]);
#pragma unroll
      for (int w = 0; w < WAVES; ++w)
        sum += s_l[w][16 * x + qr] * (top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(s_m[w][16 * x + qr] - top));
      const int i = row / G, gh = row - i * G;
      const int64_t at = (sq.first + i) * Hq + h * G + gh;
      const float inv = sum == 0.0f ? 0.0f : a.unit / sum;
      if (part == 0) {
        if (several) {
          float* ml = a.part_ml + ((int64_t)split * a.tokens * Hq + at) * 2;
          ml[0] = top;
          ml[1] = sum;
        } else if (a.lse) {
          a.lse[at] = sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
        }
      }
      if (EXACT || part * DT < D) {
        float v[DT] = {};
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
#pragma unroll
          for (int t = 0; t < DT; ++t) v[t] += s_o[(w * 16 + qr) * OS + part * DT + t];
        if (several) {
          float* po = a.part_o + ((int64_t)split * a.tokens * Hq + at) * D + part * DT;
#pragma unroll
          for (int t = 0; t < DT; ++t) po[t] = v[t];
        } else {
          uint16_t* to = a.out + at * D + part * DT;
          if constexpr (DT == 1) {
            to[0] = (uint16_t)pack_bf16x2(v[0] * inv, 0.0f);
          } else {
#pragma unroll
            for (int t = 0; t < DT; t += 2) reinterpret_cast<uint32_t*>(to)[t / 2] = pack_bf16x2(v[t] * inv, v[t + 1] * inv);
          }
        }
      }
    }
    __syncthreads();
  }
}

// Joins the splits of the rows.  P groups of DP / 4 lanes work on a row, each
// on every P-th split, 256 / (P DP / 4) rows to a workgroup; the groups meet in
// LDS.  Few splits of many rows take P = 1 (51 000 rows in 2: 16 us, 97 with a
// workgroup to each), many splits of few rows the whole workgroup.  Row tiles
// whose keys fit one split were finished by their own workgroup.
template <int DP, bool WIDE>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, int tile_rows) {
  constexpr int L = DP / 4, P = WIDE ? 256 / L : 1, R = 256 / (L * P);
  __shared__ __align__(16) float4 s_acc[WIDE ? P : 1][L];
  __shared__ float s_sum[WIDE ? P : 1];
  const int c = threadIdx.x % L, part = WIDE ? threadIdx.x / L : 0, b = blockIdx.y;
  const int H = a.pool.heads, G = a.group, Hq = H * G, D = a.pool.dim;
  const Seq sq = load_seq(a, b);
  const int e = blockIdx.x * R + (WIDE ? 0 : threadIdx.x / L);
  if (e >= (int64_t)sq.n * Hq) return;  // the whole workgroup where it meets
  const int i = e / Hq, hq = e - i * Hq, rows = sq.n * G;
  const int row0 = (i * G + hq % G) / tile_rows * tile_rows;
  const int hi = seen_hi(a, sq, (min(rows, row0 + tile_rows) - 1) / G), lo = seen_lo(a, sq, row0 / G) & ~15;
  if (hi - lo <= a.chunk) return;
  const int n = (hi - lo + a.chunk - 1) / a.chunk;
  const int64_t at = (sq.first + i) * Hq + hq, step = a.tokens * Hq;
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + at;
  float top = -INFINITY;
#pragma unroll 4
  for (int s = 0; s < n; ++s) top = fmaxf(top, ml[s * step].x);
  const float ref = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
  float4 acc = make_float4(0, 0, 0, 0);
  if (4 * c < D) {
#pragma unroll 4
    for (int s = part; s < n; s += P) {
      const float2 w = ml[s * step];
      const float4 v = *reinterpret_cast<const float4*>(a.part_o + (s * step + at) * D + 4 * c);
      const float f = __builtin_amdgcn_exp2f(w.x - ref);
      sum += w.y * f;
      acc.x += v.x * f; acc.y += v.y * f; acc.z += v.z * f; acc.w += v.w * f;
    }
  }
  if constexpr (WIDE) {
    s_acc[part][c] = acc;
    if (c == 0) s_sum[part] = sum;
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int p = 1; p < P; ++p) {
      const float4 v = s_acc[p][c];
      acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
      sum += s_sum[p];
    }
  }
  const float inv = sum == 0.0f ? 0.0f : a.unit / sum;
  if (4 * c < D)
    *reinterpret_cast<uint2*>(a.out + at * D + 4 * c) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (c == 0 && a.lse) a.lse[at] = sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

// The join's workgroups of a sequence: one to a row where the splits are many.
int64_t join_groups(const AttendProblem& p, int64_t splits) {
  const int64_t rows = (int64_t)p.max_new * p.q.heads, per = splits > 16 ? 1 : p.pool.dim <= 64 ? 16 : p.pool.dim <= 128 ? 8 : 4;
  return (rows + per - 1) / per;
}

template <int DP>
void launch_join(const AttendArgs& a, unsigned groups, int tile_rows, hipStream_t s) {
  const dim3 grid(groups, (unsigned)a.batch);
  if (a.splits > 16) hipLaunchKernelGGL((attend_join_kernel<DP, true>), grid, dim3(256), 0, s, a, tile_rows);
  else hipLaunchKernelGGL((attend_join_kernel<DP, false>), grid, dim3(256), 0, s, a, tile_rows);
}

uint32_t bf16_round_host(float f) {  // finite f
  uint32_t u;
  std::memcpy(&u, &f, 4);
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}
float bf16_value_host(uint32_t h) {
  const uint32_t u = h << 16;
  float f;
  std::memcpy(&f, &u, 4);
  return f;
}

// How a problem is cut: rows per tile, row tiles, splits of the keys and the
// keys of a split.
struct Plan {
  bool tile;  // the tile kernel, else the streaming one
  int tile_rows, waves;
  int64_t tiles, splits, chunk;
};

Plan make_plan(const AttendProblem& p) {
  Plan r{};
  const int64_t group = p.q.heads / p.pool.heads, rows = p.max_new * group;
  r.tile = rows > 32;
  // Quantized rows are widened once per tile: 256 rows share that where there
  // are more than 128; bf16 rows need none of it, and two smaller workgroups of a
  // CU overlap their matrix and vector phases.  us with 128 and 256 rows, 4
  // sequences of n tokens over 2048, 32 heads: n = 129 int8 69 64, NF4 78 69, FP4
  // 73 67; 200: 68 71, 77 76, 75 76; 250: 74 77, 81 83, 79 82; 300: 99 98, 110
  // 106, 109 106; 500: 115 111, 128 116, 125 115.  Where there are few workgroups
  // the larger tiles lose: 33 tokens of 64 heads over 8192 keys of 8, int8 40
  // 54, NF4 47 60.
  r.tile_rows = r.tile ? (rows > 128 && p.pool.type != kKVBF16 && p.pool.dim <= 128 ? 256 : 128) : rows > 16 && p.pool.dim <= 128 ? 32 : 16;
  r.tiles = std::max<int64_t>(1, (rows + r.tile_rows - 1) / r.tile_rows);
  // Keys that a tile can see (`reach`), from a multiple of 16 on where a window
  // cuts them.
  const bool cut = p.window > 0 && p.causal && (int64_t)p.window + r.tile_rows < p.max_len;
  int64_t span = (cut ? (int64_t)p.window + r.tile_rows : p.max_len) + 15;
  const int64_t reach = std::min<int64_t>(p.max_len, span);
  const int64_t work = std::max<int64_t>(1, (int64_t)p.batch * p.pool.heads * r.tiles);
  // Splits cost a second launch and its partial sums (6 us at the least).
  int64_t splits = 1;
  if (r.tile) {
    // Tiles are long and uneven (a sequence's length, the causal corner), so they
    // want twice what the chip holds at once: 4 chunks of 300 to 512 tokens over
    // 512 to 4608, int8, 173 us whole, 132 + 12 in two, 140 + 14 in three.
    const int64_t full = r.tile_rows == 256 ? 512 : 1024;
    if (work < full) splits = std::min((full + work - 1) / work, span / 256);
  } else if (work < 128) {
    // Streaming, one workgroup to a CU: 8 heads of 131071 NF4 keys 43 + 4 us in
    // 32 splits of eight waves, 44 + 5.5 in 64 of four.
    splits = std::min(256 / work, span / 512);
  } else {
    // A CU takes as long for two workgroups as for one twice as long (nearly), so
    // the fullest CU's keys count, against the join: 1000 keys' time and 500 for
    // each split's sums.  us in 1, 2, 3, 4 splits: 128 sequences and heads of 4000
    // NF4 keys 36 27 35 30 (bf16 66 55 63 57), 145 of 7324 82 88 68 74, 320 of 4000
    // 75 70 70 73, 512 of 500 to 4000 69 74 79 84, 128 of 200 to 1000, bf16, 16 17.
    int64_t least = (work + 255) / 256 * span;
    for (int64_t s = 2; s <= 4 && span / s >= 512; ++s) {
      const int64_t keys = (work * s + 255) / 256 * (span / s) + 500 * (s + 1);
      if (keys < least) {
        least = keys;
        splits = s;
      }
    }
  }
  splits = std::max<int64_t>(splits, 1);
  // Eight waves to a workgroup where each has steps enough; four for short
  // sequences (those 4 of up to 1000 tokens: 16.1 us, 17.8 with eight).
  r.waves = span / splits > 2048 && r.tile_rows == 16 && p.pool.dim <= 128 ? 8 : 4;
  r.chunk = ((span + splits - 1) / splits + 127) / 128 * 128;
  r.chunk = std::max<int64_t>(r.chunk, 128);
  if (!r.tile) r.chunk = std::min<int64_t>(r.chunk, kMaxChunk);
  r.splits = std::max<int64_t>(1, (reach + r.chunk - 1) / r.chunk);
  return r;
}

template <int KT, int DP, int NQ, int WAVES>
void stream_dim(const AttendArgs& a, unsigned grid, hipStream_t s) {
  if (a.pool.dim == DP) hipLaunchKernelGGL((attend_stream_kernel<KT, DP, NQ, WAVES, true>), dim3(grid), dim3(64 * WAVES), 0, s, a);
  else hipLaunchKernelGGL((attend_stream_kernel<KT, DP, NQ, WAVES, false>), dim3(grid), dim3(64 * WAVES), 0, s, a);
}
template <int KT, int NQ>
void stream_type(const AttendArgs& a, int waves, unsigned grid, hipStream_t s) {
  if constexpr (NQ == 2) {  // four waves, heads of up to 128 (see make_plan)
    if (a.pool.dim <= 64) stream_dim<KT, 64, 2, 4>(a, grid, s);
    else stream_dim<KT, 128, 2, 4>(a, grid, s);
  } else {
    if (a.pool.dim > 128) stream_dim<KT, 256, 1, 4>(a, grid, s);
    else if (a.pool.dim > 64) waves == 8 ? stream_dim<KT, 128, 1, 8>(a, grid, s) : stream_dim<KT, 128, 1, 4>(a, grid, s);
    else waves == 8 ? stream_dim<KT, 64, 1, 8>(a, grid, s) : stream_dim<KT, 64, 1, 4>(a, grid, s);
  }
}
template <int NQ>
void stream_rows(const AttendArgs& a, int waves, unsigned grid, hipStream_t s) {
  if (a.pool.type == kKVBF16) stream_type<kOpBF16, NQ>(a, waves, grid, s);
  else if (a.pool.type == kKVINT8) stream_type<kOpINT8, NQ>(a, waves, grid, s);
  else if (a.pool.type == kKVNF4) stream_type<kOpLevel2, NQ>(a, waves, grid, s);
  else stream_type<kOpLevel, NQ>(a, waves, grid, s);
}

}  // namespace

bool attend_fits(const AttendProblem& p) {
  // Rows and (token, head) pairs are counted in 32 bits.
  if ((int64_t)p.max_new * p.q.heads >= (int64_t(1) << 30)) return false;
  const Plan r = make_plan(p);
  const int64_t groups = (int64_t)p.batch * p.pool.heads, threads = 64 * (r.tile ? r.tile_rows / 32 : r.waves);
  if (r.tiles > INT32_MAX || groups * r.tiles > INT32_MAX || !grid_fits(groups * r.tiles * r.splits * threads)) return false;
  return r.splits == 1 || grid_fits(join_groups(p, r.splits) * 256);
}

size_t attend_workspace_bytes(const AttendProblem& p) {
  const Plan r = make_plan(p);
  if (r.splits <= 1) return 0;
  const int64_t rows = r.splits * p.tokens * p.q.heads;
  return (size_t)(rows * 2 * 4 + 255) / 256 * 256 + (size_t)rows * p.pool.dim * 4;
}

hipError_t launch_attend(const AttendProblem& p, const float table[16], void* ws, hipStream_t s) {
  AttendArgs a{};
  hipError_t e = hipSuccess;
  a.status = status_word(&e);
  if (!a.status) return e;
  const Plan r = make_plan(p);
  a.pool = p.pool;
  a.q = p.q;
  a.tokens = p.tokens;
  a.pages = p.pages;
  a.width = p.width;
  a.starts = p.starts;
  a.lengths = p.lengths;
  a.batch = p.batch;
  a.group = p.q.heads / p.pool.heads;
  a.max_new = p.max_new;
  a.max_len = p.max_len;
  a.scale2 = p.scale * kLog2e;
  a.causal = p.causal;
  a.window = p.window;
  a.out = p.out;
  a.lse = p.lse;
  a.splits = (int32_t)r.splits;
  a.chunk = (int32_t)r.chunk;
  a.tiles = (int32_t)r.tiles;
  a.unit = p.pool.type == kKVINT4 ? 1.0f / 7.0f : p.pool.type == kKVFP4 ? 1.0f / 6.0f : 1.0f;
  for (int c = 0; c < 16; ++c) {
    const float f = p.pool.type == kKVINT4 ? std::rint(table[c] * 7.0f) : p.pool.type == kKVFP4 ? std::rint(table[c] * 12.0f) / 2.0f : table[c];
    const uint32_t hi = bf16_round_host(f);
    a.levels[c] = hi | bf16_round_host(f - bf16_value_host(hi)) << 16;
    a.values[c] = table[c];
  }
  if (r.splits > 1) {
    const size_t ml = (size_t)(r.splits * p.tokens * p.q.heads * 2 * 4 + 255) / 256 * 256;
    a.part_ml = static_cast<float*>(ws);
    a.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + ml);
  }
  if (r.tile) {
    KernelTimer kt_("attend_tile_kernel", s);
    launch_attend_tile(a, r.tile_rows, s);
    e = hipGetLastError();
  } else {
    KernelTimer kt_("attend_stream_kernel", s);
    const unsigned grid = (unsigned)(p.batch * p.pool.heads * r.tiles * r.splits);
    if (r.tile_rows == 16) stream_rows<1>(a, r.waves, grid, s);
    else stream_rows<2>(a, r.waves, grid, s);
    e = hipGetLastError();
  }
  if (e != hipSuccess || r.splits == 1) return e;
  KernelTimer kt_("attend_join_kernel", s);
  const unsigned groups = (unsigned)join_groups(p, r.splits);
  if (p.pool.dim <= 64) launch_join<64>(a, groups, r.tile_rows, s);
  else if (p.pool.dim <= 128) launch_join<128>(a, groups, r.tile_rows, s);
  else launch_join<256>(a, groups, r.tile_rows, s);
  return hipGetLastError();
}

}  // namespace qlora
