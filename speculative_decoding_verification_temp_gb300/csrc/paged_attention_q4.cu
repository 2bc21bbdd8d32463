// Attention over a paged cache of 4-bit rows (q4.cuh): head_dim 64 or 128, queries and
// outputs of 16 bits, 8 or 16 rows of queries per unit (new tokens times the group's
// heads).
//
// A warp takes 32 keys of a tile of 128.  Scores: the keys are the rows of the matrix
// instruction and the queries its columns, so that up to eight rows of queries cost
// what one does.  A code n, masked out of its word and taken as float16, is the
// subnormal n 2^-24 (16 n 2^-24 for the odd nibbles, whose queries are divided by 16): the
// products are exact, and cost a mask each.  Each of the four groups of a row has sums
// of its own; a key's score is
//   sum over groups g of s_g (q . n)_g + m_g (sum of q)_g
// with the scales applied to the sums in float32 and the minima as one more step of
// the instruction, against the queries' sums in two float16 terms.  So scores are as
// exact as those of rows in float16 without any value being made.  Queries enter as
// float16, each row scaled by a power of two to 2^9 at most: exact but for what lies
// 2^-24 below a row's largest.
//
// Outputs: the values are the rows, the keys the inner dimension.  Two tokens' words are
// swapped into pairs of tokens, a nibble becomes 1024 + n or 64 + n by its mask, n by
// a subtraction and m + s n by one more instruction, rounded to float16 once (half a
// step of 2^-11, against quantisation by half a step of 1/15 of the spread).  The weights
// of 8 keys and 8 rows cross from the scores' layout to the products' by one
// transposing move.  Weights are float16 as in the tensor-memory kernels: lifted, so
// that those rounded to zero are below 2^-32 of the row's largest.
//
// One warp of the CTA copies: a bulk copy per page and head where a head's tokens lie
// one behind another, one per row elsewhere.  It runs ahead of the four others across
// the ends of units.
#include "paged_attention_wide.cuh"
#include "q4.cuh"

namespace sv {

namespace {

constexpr int kQ4Tile = 128;  // keys of a tile
constexpr int kQ4Own = 32;    // of a warp
constexpr int kSms4 = 152;
// Weights reach 2^(kLift4 + kSlack) = 2^14, and times scales below 2 stay in float16;
// larger scales lower the weights (see cap).
constexpr float kLift4 = 6.f;

template <int D, int NT>
struct Rows4 {
  static constexpr int kRow = q4_row_bytes(D);
  static constexpr int kRows = 8 * NT;
  static constexpr int kWarps = 4;                    // that compute
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kCtas = NT == 1 ? 3 : 2;       // of an SM
  static constexpr int kStages = NT == 1 ? 3 : 4;
  static constexpr int kStage = 2 * kQ4Tile * kRow;   // keys, then values
  // a lane's part of the queries: products' operands, their sums, two factors
  static constexpr int kQWords = (D / 8 + 3 + 3) / 4 * 4;
  static constexpr int kQueries = kStages * kStage;
  static constexpr int kUnits = 2 * NT * D / 32;      // 16-byte pieces of a lane's outputs
  static constexpr int kMeet = kQueries + NT * 32 * kQWords * 4;
  static constexpr int kSmem = kMeet + kWarps / 2 * kUnits * 32 * 16;
};

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                      uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The first of a sum.
__device__ __forceinline__ void mma16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma8_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t as_word(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }
__device__ __forceinline__ uint32_t word_at(const char *p) { return *reinterpret_cast<const uint32_t *>(p); }

// Two outputs of token n that the keys' values which are not finite (beyond float16
// too) add, from the parts of tiles that some row does not see whole; see
// nonfinite_values.
template <int D>
static __device__ __noinline__ float2 nonfinite_values_q4(const AttnParams &p, const UnitWalk u, int n,
                                                          int d) {
  float a[2] = {0.f, 0.f};
  for (int i = u.i0; i < u.i1; ++i) {
    const int t0 = key_tile(u.k, i) << p.tile_log2;
    for (int at0 = t0; at0 < t0 + (1 << p.tile_log2) && at0 < u.k.end; at0 += kQ4Own) {
      bool whole = all_seen(p, u.k, at0, kQ4Own);
      for (int at = at0; at < at0 + kQ4Own && whole; ++at)
        whole = at < u.k.end && page_ok(p.C, page_at(p.S, u.b, at / p.C.page_size));
      if (whole) continue;
      for (int at = at0; at < min(at0 + kQ4Own, u.k.end); ++at) {
        const int index = at / p.C.page_size, page = page_at(p.S, u.b, index);
        if (!page_ok(p.C, page) || !sees(p, u.k, u.b, n, at)) continue;
        const char *row = p.C.v + page * p.C.v_page + (at - index * p.C.page_size) * p.C.v_token +
                          u.h * p.C.v_head;
        const float2 s = q4_pair(word_at(row + D / 2 + d / (D / 4) * 4));
        if (q4_finite(s)) continue;
        float x[8];
        q4_codes(word_at(row + d / 8 * 4), x);
        for (int j = 0; j < 2; ++j) {
          const float v = fmaf(s.x, x[d % 8 + j], s.y);
          a[j] += fabsf(v) < 65520.f ? 0.f : (isnan(v) ? v : copysignf(INFINITY, v));
        }
      }
    }
  }
  return make_float2(a[0], a[1]);
}

// A lane's part of eight rows of queries, from row nt * 8 of the unit: for the products
// with the codes, row g of column g; see Rows4::kQWords.
template <class E, int D>
__device__ __forceinline__ void prepare_queries(const AttnParams &p, const UnitWalk &u, int nt, int lane,
                                                uint32_t *to) {
  using TE = typename E::T;
  constexpr int kN = D / 16;  // values of each group
  const int g = lane >> 2, t = lane & 3, live = u.live_rows(p), row = nt * 8 + g;
  const int r = u.r0 + min(row, live - 1), n = r / p.G;
  const char *q = p.q + u.b * p.q_seq + n * p.q_token + (u.h * p.G + r - n * p.G) * p.q_head;
  float x[4][kN];
  float top = 0.f;
  bool odd = false;
  uint32_t v[4][kN / 2];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const TE *from = reinterpret_cast<const TE *>(q) + j * (D / 4) + t * kN;
    if constexpr (D == 128) {
      const uint4 y = *reinterpret_cast<const uint4 *>(from);
      v[j][0] = y.x, v[j][1] = y.y, v[j][2] = y.z, v[j][3] = y.w;
    } else {
      const uint2 y = *reinterpret_cast<const uint2 *>(from);
      v[j][0] = y.x, v[j][1] = y.y;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      x[j][e] = row < live ? E::to(reinterpret_cast<const TE *>(v[j])[e]) : 0.f;
      odd |= !isfinite(x[j][e]);
      top = fmaxf(top, fabsf(x[j][e]));
    }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    odd |= __shfl_xor_sync(0xFFFFFFFFu, static_cast<int>(odd), o) != 0;
  }
  // to [2^8, 2^9); rows of zeros, and those far below what matters, stay
  const int exponent = top > 1e-30f ? min(max(8 - ilogbf(top), -126), 126) : 0;
  const float up = __int_as_float((127 + exponent) << 23);
  // a query that is not finite makes its row NaN
  const float factor = odd ? __int_as_float(0x7FC00000)
                           : p.scale_log2 * __int_as_float((127 - exponent) << 23);
  uint32_t sums = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      // as the products see it
      x[j][e] = odd ? 0.f : __half2float(__float2half_rn(x[j][e] * up));
      sum += x[j][e];
    }
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
    const __half hi = __float2half_rn(sum);
    const __half lo = __float2half_rn(sum - __half2float(hi));
    if (t == j) sums = as_word(__halves2half2(hi, lo));
#pragma unroll
    for (int s = 0; s < kN / 4; ++s) {
      to[(j * (kN / 4) + s) * 2] = F16::pack(x[j][4 * s], x[j][4 * s + 1]);
      to[(j * (kN / 4) + s) * 2 + 1] = F16::pack(x[j][4 * s + 2] * 0.0625f, x[j][4 * s + 3] * 0.0625f);
    }
  }
  to[D / 8] = sums;
  // of this lane's two columns of the scores
  to[D / 8 + 1] = __float_as_uint(__shfl_sync(0xFFFFFFFFu, factor, 2 * t * 4));
  to[D / 8 + 2] = __float_as_uint(__shfl_sync(0xFFFFFFFFu, factor, (2 * t + 1) * 4));
}

template <int kStages>
struct Rows4Ctl {
  unsigned long long full[kStages], empty[kStages], q_full, q_empty;
  alignas(16) uint32_t valid[kStages][4];
  int dead, bad;
};

}  // namespace

template <class E, int D, int NT>
__global__ void __launch_bounds__(Rows4<D, NT>::kThreads, Rows4<D, NT>::kCtas)
    rows4_kernel(const __grid_constant__ AttnParams p) {
  using L = Rows4<D, NT>;
  using TE = typename E::T;
  constexpr int kRow = L::kRow, kStages = L::kStages, R = L::kRows;
  extern __shared__ __align__(128) char smem4[];
  __shared__ Rows4Ctl<kStages> ctl;
  __shared__ RunScratch<L::kThreads, 1> runs;
  __shared__ float ml_s[L::kWarps][2][R];
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(&ctl.full[i], 1);
      bar_init(&ctl.empty[i], L::kWarps);
    }
    bar_init(&ctl.q_full, 1);
    bar_init(&ctl.q_empty, L::kWarps);
    ctl.dead = ctl.bad = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  Line lines[1];
  find_runs(p, runs, blockIdx.x, 0, lines);  // barriers as well
  const Line &line = lines[0];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  UnitWalk u;
  const bool busy = u.start(p, line);
  if (tid == 0) write_join(p, line, busy ? &u : nullptr);
  if (!busy) return;

  if (warp == L::kWarps) {
    // ------------------------------------------------------ copies and queries
    const int P = p.C.page_size;
    const bool packed_k = P == 1 || p.C.k_token == kRow, packed_v = P == 1 || p.C.v_token == kRow;
    const float per_page = 1.f / static_cast<float>(P);
    // exact below 2^21: a quotient's distance from a whole number is 1 / (2 P) at least
    auto pages_in = [&](int x) { return static_cast<int>((static_cast<float>(x) + 0.5f) * per_page); };
    uint32_t tiles = 0, units = 0;
    bool ok = true;
    do {
      // A tile's pages are slots, the lane-th of which this lane looks up (and those 32
      // and more behind it, where pages are shorter than five tokens), a tile ahead.
      auto look_up = [&](int at0, int index0, int in_page0, int slot) {
        const int at = max(at0, at0 - in_page0 + slot * P);
        // not behind the last key, nor between the sinks and the window
        if (at >= min(at0 + kQ4Tile, u.k.end)) return -1;
        if (at >= p.sinks && at0 - in_page0 + (slot + 1) * P <= u.k.first) return -1;
        return page_at(p.S, u.b, index0 + slot);
      };
      int at0 = key_tile(u.k, u.i0) * kQ4Tile, index0 = at0 / P, in_page0 = at0 - index0 * P;
      int page = look_up(at0, index0, in_page0, lane);
      for (int i = u.i0; ok && i < u.i1; ++i, ++tiles) {
        const int st = tiles % kStages;
        const int next_at0 = key_tile(u.k, i + 1) * kQ4Tile, next_index0 = next_at0 / P,
                  next_in_page0 = next_at0 - next_index0 * P;
        int next = -1;
        if (i + 1 < u.i1) next = look_up(next_at0, next_index0, next_in_page0, lane);
        if (!(ok = warp_wait(&ctl.empty[st], ((tiles / kStages) & 1u) ^ 1u, &ctl.dead))) break;
        const uint32_t stage = smem_u32(smem4) + st * L::kStage;
        const int slots = pages_in(in_page0 + kQ4Tile - 1) + 1;
        uint32_t there[4] = {0u, 0u, 0u, 0u};
        // the keys of slot s that are there: [from, to), and from `again` on, where the
        // window begins behind the sinks within the page
        auto keys_of = [&](int s, int page_id, int &from, int &to, int &again, int &end) {
          from = max(0, s * P - in_page0);
          end = min(min(kQ4Tile, (s + 1) * P - in_page0), u.k.end - at0);
          if (!page_ok(p.C, page_id)) end = from;
          to = again = end;
          if (p.sinks < u.k.first) {
            to = max(from, min(end, p.sinks - at0));
            again = min(end, max(to, u.k.first - at0));
          }
          end = max(from, end);
          to = min(max(to, from), end);
          again = min(max(again, to), end);
        };
        for (int s = lane; s < slots; s += 32) {
          int from, to, again, end;
          keys_of(s, s < 32 ? page : look_up(at0, index0, in_page0, s), from, to, again, end);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            there[w] |= low_bits(to - 32 * w) & ~low_bits(from - 32 * w);
            there[w] |= low_bits(end - 32 * w) & ~low_bits(again - 32 * w);
          }
        }
        int count = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          there[w] = __reduce_or_sync(0xFFFFFFFFu, there[w]);
          count += __popc(there[w]);
        }
        if (lane == 0) {
          *reinterpret_cast<uint4 *>(ctl.valid[st]) = make_uint4(there[0], there[1], there[2], there[3]);
          bar_expect(&ctl.full[st], 2 * kRow * count);
        }
        __syncwarp();
        for (int s = lane; s < slots; s += 32) {
          int from, to, again, end;
          const int id = s < 32 ? page : look_up(at0, index0, in_page0, s);
          keys_of(s, id, from, to, again, end);
          if (!page_ok(p.C, id)) continue;
          // the page's token at key 0 of the tile
          const long long token0 = static_cast<long long>(in_page0) - static_cast<long long>(s) * P;
          auto copy = [&](bool packed, uint32_t to_s, const char *base, long long token, int a, int b) {
            if (a >= b) return;
            if (packed) {
              bulk_load(to_s + a * kRow, base + (token0 + a) * token, (b - a) * kRow, &ctl.full[st]);
            } else {
              for (int key = a; key < b; ++key)
                bulk_load(to_s + key * kRow, base + (token0 + key) * token, kRow, &ctl.full[st]);
            }
          };
          const char *k = p.C.k + id * p.C.k_page + u.h * p.C.k_head, *v = p.C.v + id * p.C.v_page + u.h * p.C.v_head;
          copy(packed_k, stage, k, p.C.k_token, from, to);
          copy(packed_v, stage + kQ4Tile * kRow, v, p.C.v_token, from, to);
          copy(packed_k, stage, k, p.C.k_token, again, end);
          copy(packed_v, stage + kQ4Tile * kRow, v, p.C.v_token, again, end);
        }
        __syncwarp();
        if (tiles == 0) first_wait(&ctl.full[0], p.first_wait, &ctl.dead);
        if (i == u.i0) {
          // the unit's queries, behind the copies of its first tile and once those of the
          // unit before have been taken
          if (!(ok = warp_wait(&ctl.q_empty, (units & 1u) ^ 1u, &ctl.dead))) {
            ++tiles;
            break;
          }
          ++units;
          for (int nt = 0; nt < NT; ++nt)
            prepare_queries<E, D>(p, u, nt, lane,
                                  reinterpret_cast<uint32_t *>(smem4 + L::kQueries) +
                                      (nt * 32 + lane) * L::kQWords);
          __syncwarp();
          if (lane == 0) bar_arrive(&ctl.q_full);
        }
        at0 = next_at0;
        index0 = next_index0;
        in_page0 = next_in_page0;
        page = next;
      }
    } while (ok && u.next(p, line));
    // no copy is in flight when the CTA ends
    for (uint32_t i = tiles > kStages ? tiles - kStages : 0; i < tiles; ++i)
      bar_linger(&ctl.full[i % kStages], (i / kStages) & 1u);
  } else {
    // -------------------------------------------------------------- products
    const int g = lane >> 2, t = lane & 3;
    constexpr int kSteps = D / 16;   // of the scores' products
    constexpr int kOuts = D / 16;    // 16 dimensions each of the outputs
    // bytes of two tokens' words: this lane's codes of the even dimensions, the odd ones
    const int byte = D == 128 ? g & 1 : (g >> 1) & 1;
    // (the halves' upper bytes are whatever byte 0 is, and masked out below)
    const uint32_t sel_even = byte | (4 + byte) << 8, sel_odd = (2 + byte) | (6 + byte) << 8;
    const uint32_t nibble = D == 64 && (g & 1) ? 0x00F000F0u : 0x000F000Fu;
    uint32_t tiles = 0, units = 0;
    do {
      uint32_t qf[NT][kSteps][2], qs[NT];
      float c[NT][2];
      const int live = u.live_rows(p);
      warp_wait(&ctl.q_full, units++ & 1u, &ctl.dead);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t x[L::kQWords];
        const uint4 *from = reinterpret_cast<const uint4 *>(smem4 + L::kQueries) +
                            (nt * 32 + lane) * (L::kQWords / 4);
#pragma unroll
        for (int i = 0; i < L::kQWords / 4; ++i) {
          const uint4 y = from[i];
          x[4 * i] = y.x, x[4 * i + 1] = y.y, x[4 * i + 2] = y.z, x[4 * i + 3] = y.w;
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) qf[nt][s][0] = x[2 * s], qf[nt][s][1] = x[2 * s + 1];
        qs[nt] = x[D / 8];
        c[nt][0] = __uint_as_float(x[D / 8 + 1]);
        c[nt][1] = __uint_as_float(x[D / 8 + 2]);
      }
      __syncwarp();
      if (lane == 0) bar_arrive(&ctl.q_empty);
      float m[NT][2], l[NT][2], o[NT][kOuts][4], om[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
        om[nt][0] = om[nt][1] = om[nt][2] = om[nt][3] = 0.f;
#pragma unroll
        for (int i = 0; i < kOuts; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      }
      // scales are below 2^(cap + 1)
      int cap = 0;

      for (int i = u.i0; i < u.i1; ++i, ++tiles) {
        const int st = tiles % kStages;
        // a wait that gave up: the tiles go on uncounted, so that the warps meet at the
        // units' ends
        if (!warp_wait(&ctl.full[st], (tiles / kStages) & 1u, &ctl.dead)) continue;
        const int at0 = key_tile(u.k, i) * kQ4Tile + warp * kQ4Own;
        const uint32_t valid = ctl.valid[st][warp];
        char *k_s = smem4 + st * L::kStage + warp * kQ4Own * kRow, *v_s = k_s + kQ4Tile * kRow;
        if (valid != 0u) {
          float y[2][NT][4];
#pragma unroll
          for (int blk = 0; blk < 2; ++blk) {
            const char *r0 = k_s + (blk * 16 + g) * kRow, *r1 = r0 + 8 * kRow;
            float a[NT][4][4], am[NT][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if constexpr (D == 128) {
                const uint32_t x0 = word_at(r0 + j * 16 + t * 4), x1 = word_at(r1 + j * 16 + t * 4);
                const uint32_t z0 = x0 >> 8, z1 = x1 >> 8;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  mma16_first(a[nt][j], x0 & 0x000F000Fu, x1 & 0x000F000Fu, x0 & 0x00F000F0u,
                              x1 & 0x00F000F0u, qf[nt][2 * j][0], qf[nt][2 * j][1]);
                  mma16(a[nt][j], z0 & 0x000F000Fu, z1 & 0x000F000Fu, z0 & 0x00F000F0u,
                        z1 & 0x00F000F0u, qf[nt][2 * j + 1][0], qf[nt][2 * j + 1][1]);
                }
              } else {
                const int shift = (t & 1) * 8;
                const uint32_t x0 = word_at(r0 + j * 8 + (t >> 1) * 4) >> shift;
                const uint32_t x1 = word_at(r1 + j * 8 + (t >> 1) * 4) >> shift;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma16_first(a[nt][j], x0 & 0x000F000Fu, x1 & 0x000F000Fu, x0 & 0x00F000F0u,
                              x1 & 0x00F000F0u, qf[nt][j][0], qf[nt][j][1]);
              }
            }
            const uint4 s0 = *reinterpret_cast<const uint4 *>(r0 + D / 2);
            const uint4 s1 = *reinterpret_cast<const uint4 *>(r1 + D / 2);
            const uint32_t m0 = __byte_perm(word_at(r0 + D / 2 + t * 4), 0, 0x3232);
            const uint32_t m1 = __byte_perm(word_at(r1 + D / 2 + t * 4), 0, 0x3232);
            const float f0[4] = {__low2float(as_half2(s0.x)), __low2float(as_half2(s0.y)),
                                 __low2float(as_half2(s0.z)), __low2float(as_half2(s0.w))};
            const float f1[4] = {__low2float(as_half2(s1.x)), __low2float(as_half2(s1.y)),
                                 __low2float(as_half2(s1.z)), __low2float(as_half2(s1.w))};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma8_first(am[nt], m0, m1, qs[nt]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float *f = e < 2 ? f0 : f1;
                const float z = fmaf(f[3], a[nt][3][e],
                                     fmaf(f[2], a[nt][2][e], fmaf(f[1], a[nt][1][e], f[0] * a[nt][0][e])));
                y[blk][nt][e] = fmaf(z, 16777216.f, am[nt][e]) * c[nt][e & 1];
              }
            }
          }
          // this lane's key: its values' scales
          uint4 *scales = reinterpret_cast<uint4 *>(v_s + lane * kRow + D / 2);
          uint4 s = *scales;
          if (valid != 0xFFFFFFFFu || !all_seen(p, u.k, at0, kQ4Own)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int n = (u.r0 + min(nt * 8 + 2 * t + e, live - 1)) / p.G;
#pragma unroll
                for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const int key = blk * 16 + h * 8 + g;
                    if (!((valid >> key) & 1u) || !sees(p, u.k, u.b, n, at0 + key))
                      y[blk][nt][2 * h + e] = -INFINITY;
                  }
              }
            // rows that were not copied stand for zeros, and so do groups that are not
            // finite, which nonfinite_values_q4 adds
            uint32_t *w = reinterpret_cast<uint32_t *>(&s);
            const bool there = (valid >> lane) & 1u;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (!there || !q4_finite(q4_pair(w[j]))) {
                if (there) *reinterpret_cast<volatile int *>(&ctl.bad) = 1;
                w[j] = 0u;
              }
            *scales = s;
            __syncwarp();
          }
          // scales of 2^(cap + 1) and more: the weights are lowered
          if (__any_sync(0xFFFFFFFFu, ((s.x | s.y) | (s.z | s.w)) & 0x4000u)) {
            const uint32_t top = max(max(s.x & 0x7FFFu, s.y & 0x7FFFu), max(s.z & 0x7FFFu, s.w & 0x7FFFu));
            const uint32_t finite = __reduce_max_sync(0xFFFFFFFFu, top < 0x7C00u ? top : 0u);
            const int more = static_cast<int>(finite >> 10) - 15 - cap;
            if (more > 0) {
              cap += more;
              const float f = __int_as_float((127 - more) << 23);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  m[nt][e] += static_cast<float>(more);
                  l[nt][e] *= f;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  om[nt][e] *= f;
#pragma unroll
                  for (int j = 0; j < kOuts; ++j) o[nt][j][e] *= f;
                }
              }
            }
          }
          // the running maximum
          const float lift = kLift4 - static_cast<float>(cap);
          bool up = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float top = fmaxf(fmaxf(y[0][nt][e], y[0][nt][2 + e]), fmaxf(y[1][nt][e], y[1][nt][2 + e]));
              up |= top - lift > m[nt][e] + kSlack;
            }
          if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float top = fmaxf(fmaxf(y[0][nt][e], y[0][nt][2 + e]), fmaxf(y[1][nt][e], y[1][nt][2 + e]));
#pragma unroll
                for (int s = 4; s <= 16; s <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
                top -= lift;
                const float to = top > m[nt][e] + kSlack ? top : m[nt][e];
                const float f = m[nt][e] == -INFINITY ? 0.f : fast_exp2(m[nt][e] - to);
                m[nt][e] = to;
                l[nt][e] *= f;
                om[nt][e] *= f;
#pragma unroll
                for (int j = 0; j < kOuts; ++j) {
                  o[nt][j][e] *= f;
                  o[nt][j][2 + e] *= f;
                }
              }
          }
          uint32_t w[2][NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            // a row that has seen nothing yet keeps weights of zero
            const float u0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], u1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
            for (int blk = 0; blk < 2; ++blk)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float p0 = fast_exp2(y[blk][nt][2 * h] - u0), p1 = fast_exp2(y[blk][nt][2 * h + 1] - u1);
                l[nt][0] += p0;
                l[nt][1] += p1;
                w[blk][nt][h] = transposed(F16::pack(p0, p1));
              }
          }
#pragma unroll
          for (int blk = 0; blk < 2; ++blk) {
            // tokens 2t, 2t + 1 of the first eight keys (h = 0) and of the second
            const char *v0 = v_s + (blk * 16 + 2 * t) * kRow;
            uint32_t sp[2][4], mp[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const char *va = v0 + h * 8 * kRow + D / 2, *vb = va + kRow;
              const uint4 pa = *reinterpret_cast<const uint4 *>(va), pb = *reinterpret_cast<const uint4 *>(vb);
              sp[h][0] = __byte_perm(pa.x, pb.x, 0x5410);
              sp[h][1] = __byte_perm(pa.y, pb.y, 0x5410);
              sp[h][2] = __byte_perm(pa.z, pb.z, 0x5410);
              sp[h][3] = __byte_perm(pa.w, pb.w, 0x5410);
              // of group g mod 4; the products' other rows are not looked at
              mp[h] = __byte_perm(word_at(va + (g & 3) * 4), word_at(vb + (g & 3) * 4), 0x7632);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16(om[nt], mp[0], 0u, mp[1], 0u, w[blk][nt][0], w[blk][nt][1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t a[4];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const char *at = v0 + h * 8 * kRow + j * (D / 8) + (D == 128 ? g >> 1 : g >> 2) * 4;
                const uint32_t xa = word_at(at), xb = word_at(at + kRow);
                a[2 * h] = __byte_perm(xa, xb, sel_even);
                a[2 * h + 1] = __byte_perm(xa, xb, sel_odd);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint32_t b0 = as_word(__hmul2(as_half2(w[blk][nt][0]), as_half2(sp[0][j])));
                const uint32_t b1 = as_word(__hmul2(as_half2(w[blk][nt][1]), as_half2(sp[1][j])));
                if constexpr (D == 128) {
                  mma16(o[nt][2 * j], a[0] & 0x000F000Fu, a[1] & 0x000F000Fu, a[2] & 0x000F000Fu,
                        a[3] & 0x000F000Fu, b0, b1);
                  mma16(o[nt][2 * j + 1], a[0] & 0x00F000F0u, a[1] & 0x00F000F0u, a[2] & 0x00F000F0u,
                        a[3] & 0x00F000F0u, b0, b1);
                } else {
                  mma16(o[nt][j], a[0] & nibble, a[1] & nibble, a[2] & nibble, a[3] & nibble, b0, b1);
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&ctl.empty[st]);
      }

      // the unit's end.  Outputs as 16-byte pieces [nt][e][..]: row nt * 8 + 2t + e,
      // D 128: dimensions 32 j + 4 g .. + 3, D 64: 32 j + 2 g, + 1 and the same + 16
      float4 v[L::kUnits];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int s = 4; s <= 16; s <<= 1) l[nt][e] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][e], s);
          float low[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) low[j] = __shfl_sync(0xFFFFFFFFu, om[nt][e], j * 4 + t);
          float4 *to = v + (nt * 2 + e) * (D / 32);
          if constexpr (D == 128) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              to[j] = make_float4(fmaf(o[nt][2 * j][e], 16777216.f, low[j]),
                                  fmaf(o[nt][2 * j][2 + e], 16777216.f, low[j]),
                                  fmaf(o[nt][2 * j + 1][e], 1048576.f, low[j]),
                                  fmaf(o[nt][2 * j + 1][2 + e], 1048576.f, low[j]));
          } else {
            const float f = g & 1 ? 1048576.f : 16777216.f;
#pragma unroll
            for (int j = 0; j < 4; j += 2)
              to[j / 2] = make_float4(fmaf(o[nt][j][e], f, low[j]), fmaf(o[nt][j][2 + e], f, low[j]),
                                      fmaf(o[nt][j + 1][e], f, low[j + 1]),
                                      fmaf(o[nt][j + 1][2 + e], f, low[j + 1]));
          }
        }
      float4 *meet = reinterpret_cast<float4 *>(smem4 + L::kMeet);
      auto sums = [&] {
        if (g == 0) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              ml_s[warp][0][nt * 8 + 2 * t + e] = m[nt][e];
              ml_s[warp][1][nt * 8 + 2 * t + e] = l[nt][e];
            }
        }
      };
      auto put = [&] {
#pragma unroll
        for (int x = 0; x < L::kUnits; ++x) meet[((warp & 1) * L::kUnits + x) * 32 + lane] = v[x];
      };
      auto barrier = [&] { asm volatile("bar.sync 1, %0;" ::"n"(32 * L::kWarps) : "memory"); };
      // two warps into the two others, lane by lane
      if (warp >= 2) {
        sums();
        put();
      }
      barrier();
      if (warp < 2) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = nt * 8 + 2 * t + e;
            const float m1 = ml_s[warp + 2][0][row], l1 = ml_s[warp + 2][1][row];
            const float M = fmaxf(m[nt][e], m1);
            // a part is empty where its sum is zero: one of NaN scores has m -infinity too
            const float f0 = l[nt][e] == 0.f ? 0.f : fast_exp2(m[nt][e] - M);
            const float f1 = l1 == 0.f ? 0.f : fast_exp2(m1 - M);
            const bool none0 = l[nt][e] == 0.f, none1 = l1 == 0.f;
            m[nt][e] = M;
            l[nt][e] = (none0 ? 0.f : f0 * l[nt][e]) + (none1 ? 0.f : f1 * l1);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
              const int x = (nt * 2 + e) * (D / 32) + j;
              const float4 y = meet[((warp & 1) * L::kUnits + x) * 32 + lane];
              v[x].x = (none0 ? 0.f : f0 * v[x].x) + (none1 ? 0.f : f1 * y.x);
              v[x].y = (none0 ? 0.f : f0 * v[x].y) + (none1 ? 0.f : f1 * y.y);
              v[x].z = (none0 ? 0.f : f0 * v[x].z) + (none1 ? 0.f : f1 * y.z);
              v[x].w = (none0 ? 0.f : f0 * v[x].w) + (none1 ? 0.f : f1 * y.w);
            }
          }
        sums();
        put();
      }
      barrier();
      const bool whole = u.whole(), odd_values = *reinterpret_cast<volatile int *>(&ctl.bad) != 0;
      float *slot = p.part + piece_slot(u, line.worker) * slot_floats(p.rows, D);
      for (int x = warp; x < L::kUnits; x += L::kWarps) {
        const int row = x / (2 * (D / 32)) * 8 + 2 * t + x / (D / 32) % 2, j = x % (D / 32);
        if (row >= live) continue;
        float M = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < 2; ++w) M = fmaxf(M, ml_s[w][0][row]);
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (ml_s[w][1][row] == 0.f) continue;
          const float f = fast_exp2(ml_s[w][0][row] - M);
          const float4 z = meet[(w * L::kUnits + x) * 32 + lane];
          sum += f * ml_s[w][1][row];
          y.x += f * z.x;
          y.y += f * z.y;
          y.z += f * z.z;
          y.w += f * z.w;
        }
        const int d0 = D == 128 ? 32 * j + 4 * g : 32 * j + 2 * g, d1 = d0 + (D == 128 ? 2 : 16);
        if (odd_values) {
          const int n = (u.r0 + row) / p.G;
          const float2 z0 = nonfinite_values_q4<D>(p, u, n, d0), z1 = nonfinite_values_q4<D>(p, u, n, d1);
          y.x += z0.x, y.y += z0.y, y.z += z1.x, y.w += z1.y;
        }
        if (whole) {
          const long long at = out_row(p, u.b, u.h, u.r0 + row);
          const float n = sum == 0.f ? 0.f : 1.f / sum;
          uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<TE *>(p.out) + at * D);
          const uint32_t a = E::pack(y.x * n, y.y * n), b = E::pack(y.z * n, y.w * n);
          if constexpr (D == 128) {
            *reinterpret_cast<uint2 *>(out + d0 / 2) = make_uint2(a, b);
          } else {
            out[d0 / 2] = a;
            out[d1 / 2] = b;
          }
          if (d0 == 0 && p.lse) p.lse[at] = row_lse(M, sum);
        } else {
          float *to = slot + slot_stats(p.rows) + static_cast<size_t>(row) * D;
          *reinterpret_cast<float2 *>(to + d0) = make_float2(y.x, y.y);
          *reinterpret_cast<float2 *>(to + d1) = make_float2(y.z, y.w);
          if (d0 == 0) {
            slot[row] = M;
            slot[p.rows + row] = sum;
          }
        }
      }
      barrier();
    } while (u.next(p, line));
  }
  __syncthreads();
  if (ctl.dead) void_run<E, D, L::kThreads>(p, line);
}

namespace {

template <class E, int D, int NT>
cudaError_t start4(const AttnParams &p, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  using L = Rows4<D, NT>;
  return launch_large(rows4_kernel<E, D, NT>, done, L::kSmem, p.workers, L::kThreads, L::kSmem, stream, p);
}
template <int NT>
cudaError_t start4(const AttnParams &p, int dtype, cudaStream_t stream) {
  if (dtype == SPEC_BF16)
    return p.D == 64 ? start4<Bf16, 64, NT>(p, stream) : start4<Bf16, 128, NT>(p, stream);
  return p.D == 64 ? start4<F16, 64, NT>(p, stream) : start4<F16, 128, NT>(p, stream);
}

AttnPlan q4_plan(int N, int G) {
  if (N * G <= 8) return {Rows4<128, 1>::kCtas * kSms4, 8, 7, 1, 4};
  return {Rows4<128, 2>::kCtas * kSms4, 16, 7, 1, 4};
}

}  // namespace

size_t attention_q4_workspace_bytes(int N, int G, int D) { return plan_bytes(q4_plan(N, G), D); }

cudaError_t launch_attention_q4(AttnParams &p, int dtype, void *workspace, cudaStream_t stream) {
  take_plan(p, q4_plan(p.S.N, p.G), workspace);
  const int tiles = (p.S.N * p.G + p.rows - 1) / p.rows;
  if (p.mask && tiles <= 8) p.row_lines = tiles;
  const cudaError_t e = p.rows == 8 ? start4<1>(p, dtype, stream) : start4<2>(p, dtype, stream);
  if (e != cudaSuccess || p.whole) return e;
  return launch_join(p, dtype, stream);
}

}  // namespace sv
