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

constexpr int kQ4Warps = 4;                          // that compute
constexpr int kQ4Threads = 32 * (kQ4Warps + 1);
constexpr int kQ4Tile = 128, kQ4Own = kQ4Tile / kQ4Warps;  // keys of a tile, of a warp
constexpr int kSms4 = 152;

template <int D, int NT>
struct Rows4 {
  static constexpr int kRow = q4_row_bytes(D);
  static constexpr int kRows = 8 * NT;
  static constexpr int kStages = NT == 1 ? 3 : 4;
  static constexpr int kCtas = NT == 1 ? 3 : 2;  // of an SM
  static constexpr int kStage = 2 * kQ4Tile * kRow;  // keys, then values
  static constexpr int kMeet = kStages * kStage;     // half of the outputs of each warp
  static constexpr int kMeetFloats = kRows * D / 2;
  static constexpr int kSmem = kMeet + kQ4Warps * kMeetFloats * 4;
};

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                      uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(b0));
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t as_word(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }

// Four outputs of token n that the keys' values which are not finite (beyond float16
// too) add, from the parts of tiles that some row does not see whole; see
// nonfinite_values.
template <int D>
static __device__ __noinline__ float4 nonfinite_values_q4(const AttnParams &p, const UnitWalk u, int n,
                                                          int d, float4 acc) {
  float *a = reinterpret_cast<float *>(&acc);
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
        const float2 s = q4_pair(*reinterpret_cast<const uint32_t *>(row + D / 2 + d / (D / 4) * 4));
        float x[8];
        q4_codes(*reinterpret_cast<const uint32_t *>(row + d / 8 * 4), x);
        if (q4_finite(s)) continue;
        for (int j = 0; j < 4; ++j) {
          const float v = fmaf(s.x, x[d % 8 + j], s.y);
          a[j] += fabsf(v) < 65520.f ? 0.f : (isnan(v) ? v : copysignf(INFINITY, v));
        }
      }
    }
  }
  return acc;
}

struct Rows4Ctl {
  unsigned long long full[4], empty[4];
  alignas(16) uint32_t valid[4][4];
  RunScratch<kQ4Threads, 1> runs;
  int dead, bad;
};

}  // namespace

template <class E, int D, int NT>
__global__ void __launch_bounds__(kQ4Threads, Rows4<D, NT>::kCtas)
    rows4_kernel(const __grid_constant__ AttnParams p) {
  using L = Rows4<D, NT>;
  using TE = typename E::T;
  constexpr int kRow = L::kRow, kStages = L::kStages, R = L::kRows;
  extern __shared__ __align__(128) char smem4[];
  __shared__ Rows4Ctl ctl;
  __shared__ float ml_s[kQ4Warps][2][R];
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(&ctl.full[i], 1);
      bar_init(&ctl.empty[i], kQ4Warps);
    }
    ctl.dead = ctl.bad = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  Line lines[1];
  find_runs(p, ctl.runs, blockIdx.x, 0, lines);  // barriers as well
  const Line &line = lines[0];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  UnitWalk u;
  const bool busy = u.start(p, line);
  if (tid == 0) write_join(p, line, busy ? &u : nullptr);
  if (!busy) return;

  if (warp == kQ4Warps) {
    // ---------------------------------------------------------------- copies
    const bool packed_k = p.C.page_size == 1 || p.C.k_token == kRow;
    const bool packed_v = p.C.page_size == 1 || p.C.v_token == kRow;
    uint32_t tiles = 0;
    bool ok = true;
    do {
      for (int i = u.i0; ok && i < u.i1; ++i, ++tiles) {
        const int st = tiles % kStages;
        const int at0 = key_tile(u.k, i) * kQ4Tile;
        // this lane's tokens are at0 + lane + 32 w
        int page[4], in_page[4];
        uint32_t there[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int at = at0 + w * 32 + lane;
          page[w] = -1;
          in_page[w] = 0;
          // not behind the last key, nor between the sinks and the window
          if (at < u.k.end && (at < p.sinks || at >= u.k.first)) {
            const int index = at / p.C.page_size;
            in_page[w] = at - index * p.C.page_size;
            page[w] = page_at(p.S, u.b, index);
          }
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) there[w] = __ballot_sync(0xFFFFFFFFu, page_ok(p.C, page[w]));
        if (!(ok = warp_wait(&ctl.empty[st], ((tiles / kStages) & 1u) ^ 1u, &ctl.dead))) break;
        if (lane == 0) {
          *reinterpret_cast<uint4 *>(ctl.valid[st]) = make_uint4(there[0], there[1], there[2], there[3]);
          bar_expect(&ctl.full[st], 2 * kRow * (__popc(there[0]) + __popc(there[1]) + __popc(there[2]) +
                                                __popc(there[3])));
        }
        __syncwarp();
        const uint32_t stage = smem_u32(smem4) + st * L::kStage;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          if (!((there[w] >> lane) & 1u)) continue;
          const int key = w * 32 + lane;
          // a page's tokens are there or not together, but for the ends of what is seen:
          // its first one that is copies those behind it
          int run = 1;
          const bool packed = packed_k || packed_v;
          bool first = true;
          if (packed) {
            first = in_page[w] == 0 || key == 0 || (at0 + key == u.k.first && p.sinks < u.k.first);
            if (first) {
              run = min(p.C.page_size - in_page[w], min(kQ4Tile - key, u.k.end - at0 - key));
              // the sinks may end within a page
              if (at0 + key < p.sinks && at0 + key + run > p.sinks && p.sinks < u.k.first)
                run = p.sinks - at0 - key;
            }
          }
          const char *k = p.C.k + page[w] * p.C.k_page + in_page[w] * p.C.k_token + u.h * p.C.k_head;
          const char *v = p.C.v + page[w] * p.C.v_page + in_page[w] * p.C.v_token + u.h * p.C.v_head;
          if (!packed_k || first)
            bulk_load(stage + key * kRow, k, (packed_k ? run : 1) * kRow, &ctl.full[st]);
          if (!packed_v || first)
            bulk_load(stage + (kQ4Tile + key) * kRow, v, (packed_v ? run : 1) * kRow, &ctl.full[st]);
        }
        if (tiles == 0) first_wait(&ctl.full[0], p.first_wait, &ctl.dead);
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
    uint32_t tiles = 0;
    do {
      // this lane's part of query row g of each eight, the rows' factors
      uint32_t qf[NT][kSteps][2], qs[NT];
      float c[NT][2];
      const int live = u.live_rows(p);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int row = nt * 8 + g;
        float x[4][D / 16];  // D 128: 8 values of each group, 64: 4
        float top = 0.f;
        bool odd = false;
        const int r = u.r0 + min(row, live - 1), n = r / p.G;
        const char *q = p.q + u.b * p.q_seq + n * p.q_token + (u.h * p.G + r - n * p.G) * p.q_head;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const TE *from = reinterpret_cast<const TE *>(q) + j * (D / 4) + t * (D / 16);
          uint32_t v[D / 32];
          if constexpr (D == 128) {
            const uint4 y = *reinterpret_cast<const uint4 *>(from);
            v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2 *>(from);
            v[0] = y.x, v[1] = y.y;
          }
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {
            const TE *h = reinterpret_cast<const TE *>(v);
            x[j][e] = row < live ? E::to(h[e]) : 0.f;
            odd |= !isfinite(x[j][e]);
            top = fmaxf(top, fabsf(x[j][e]));
          }
        }
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
          odd |= __shfl_xor_sync(0xFFFFFFFFu, static_cast<int>(odd), o) != 0;
        }
        // to [2^8, 2^9) ; rows of zeros, and those far below what matters, stay
        const int exponent = top > 1e-30f ? min(max(8 - ilogbf(top), -126), 126) : 0;
        const float up = __int_as_float((127 + exponent) << 23);
        // the rows' factors of this lane's two columns; a query that is not finite makes
        // its row NaN
        const float mine = odd ? __int_as_float(0x7FC00000)
                               : p.scale_log2 * __int_as_float((127 - exponent) << 23);
        c[nt][0] = __shfl_sync(0xFFFFFFFFu, mine, 2 * t * 4);
        c[nt][1] = __shfl_sync(0xFFFFFFFFu, mine, (2 * t + 1) * 4);
        qs[nt] = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {
            // as the products see it
            x[j][e] = odd ? 0.f : __half2float(__float2half_rn(x[j][e] * up));
            sum += x[j][e];
          }
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
          const __half hi = __float2half_rn(sum);
          const __half lo = __float2half_rn(sum - __half2float(hi));
          if (t == j) qs[nt] = as_word(__halves2half2(hi, lo));
#pragma unroll
          for (int s = 0; s < D / 64; ++s) {
            qf[nt][j * (D / 64) + s][0] = F16::pack(x[j][4 * s], x[j][4 * s + 1]);
            qf[nt][j * (D / 64) + s][1] = F16::pack(x[j][4 * s + 2] * 0.0625f, x[j][4 * s + 3] * 0.0625f);
          }
        }
      }
      float m[NT][2], l[NT][2], o[NT][kOuts][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < kOuts; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      }
      int token[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) token[nt][e] = (u.r0 + min(nt * 8 + 2 * t + e, live - 1)) / p.G;

      for (int i = u.i0; i < u.i1; ++i, ++tiles) {
        const int st = tiles % kStages;
        // a wait that gave up: the tiles go on uncounted, so that the warps meet at the
        // units' ends
        if (!warp_wait(&ctl.full[st], (tiles / kStages) & 1u, &ctl.dead)) continue;
        const int at0 = key_tile(u.k, i) * kQ4Tile + warp * kQ4Own;
        const uint32_t valid = ctl.valid[st][warp];
        const bool masked = valid != 0xFFFFFFFFu || !all_seen(p, u.k, at0, kQ4Own);
        const char *k_s = smem4 + st * L::kStage + warp * kQ4Own * kRow, *v_s = k_s + kQ4Tile * kRow;
        if (valid != 0u) {
          float y[2][NT][4];
#pragma unroll
          for (int blk = 0; blk < 2; ++blk) {
            const char *r0 = k_s + (blk * 16 + g) * kRow, *r1 = r0 + 8 * kRow;
            float a[NT][4][4], am[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              am[nt][0] = am[nt][1] = am[nt][2] = am[nt][3] = 0.f;
#pragma unroll
              for (int j = 0; j < 4; ++j) a[nt][j][0] = a[nt][j][1] = a[nt][j][2] = a[nt][j][3] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if constexpr (D == 128) {
                uint32_t x0 = *reinterpret_cast<const uint32_t *>(r0 + j * 16 + t * 4);
                uint32_t x1 = *reinterpret_cast<const uint32_t *>(r1 + j * 16 + t * 4);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
                    mma16(a[nt][j], x0 & 0x000F000Fu, x1 & 0x000F000Fu, x0 & 0x00F000F0u,
                          x1 & 0x00F000F0u, qf[nt][2 * j + s][0], qf[nt][2 * j + s][1]);
                  x0 >>= 8;
                  x1 >>= 8;
                }
              } else {
                const int shift = (t & 1) * 8;
                const uint32_t x0 = *reinterpret_cast<const uint32_t *>(r0 + j * 8 + (t >> 1) * 4) >> shift;
                const uint32_t x1 = *reinterpret_cast<const uint32_t *>(r1 + j * 8 + (t >> 1) * 4) >> shift;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma16(a[nt][j], x0 & 0x000F000Fu, x1 & 0x000F000Fu, x0 & 0x00F000F0u,
                        x1 & 0x00F000F0u, qf[nt][j][0], qf[nt][j][1]);
              }
            }
            const uint4 s0 = *reinterpret_cast<const uint4 *>(r0 + D / 2);
            const uint4 s1 = *reinterpret_cast<const uint4 *>(r1 + D / 2);
            const uint32_t m0 = __byte_perm(*reinterpret_cast<const uint32_t *>(r0 + D / 2 + t * 4), 0, 0x3232);
            const uint32_t m1 = __byte_perm(*reinterpret_cast<const uint32_t *>(r1 + D / 2 + t * 4), 0, 0x3232);
            const float f0[4] = {__low2float(as_half2(s0.x)), __low2float(as_half2(s0.y)),
                                 __low2float(as_half2(s0.z)), __low2float(as_half2(s0.w))};
            const float f1[4] = {__low2float(as_half2(s1.x)), __low2float(as_half2(s1.y)),
                                 __low2float(as_half2(s1.z)), __low2float(as_half2(s1.w))};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma8(am[nt], m0, m1, qs[nt]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float *f = e < 2 ? f0 : f1;
                const float z = fmaf(f[3], a[nt][3][e],
                                     fmaf(f[2], a[nt][2][e], fmaf(f[1], a[nt][1][e], f[0] * a[nt][0][e])));
                y[blk][nt][e] = fmaf(z, 16777216.f, am[nt][e]) * c[nt][e & 1];
              }
            }
          }
          if (masked) {
#pragma unroll
            for (int blk = 0; blk < 2; ++blk)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int key = blk * 16 + h * 8 + g;
                const bool there = (valid >> key) & 1u;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    if (!there || !sees(p, u.k, u.b, token[nt][e], at0 + key))
                      y[blk][nt][2 * h + e] = -INFINITY;
              }
          }
          // the running maximum
          bool up = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float top = fmaxf(fmaxf(y[0][nt][e], y[0][nt][2 + e]), fmaxf(y[1][nt][e], y[1][nt][2 + e]));
              up |= top - kLift > m[nt][e] + kSlack;
            }
          if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float top = fmaxf(fmaxf(y[0][nt][e], y[0][nt][2 + e]), fmaxf(y[1][nt][e], y[1][nt][2 + e]));
#pragma unroll
                for (int s = 4; s <= 16; s <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
                top -= kLift;
                const float to = top > m[nt][e] + kSlack ? top : m[nt][e];
                const float f = m[nt][e] == -INFINITY ? 0.f : fast_exp2(m[nt][e] - to);
                m[nt][e] = to;
                l[nt][e] *= f;
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
            // tokens 2t, 2t + 1 of the first eight keys and of the second
            const char *v0 = v_s + (blk * 16 + 2 * t) * kRow;
            __half2 sp[2], mp[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t pa = *reinterpret_cast<const uint32_t *>(v0 + h * 8 * kRow + D / 2 + (g >> 1) * 4);
              uint32_t pb = *reinterpret_cast<const uint32_t *>(v0 + (h * 8 + 1) * kRow + D / 2 + (g >> 1) * 4);
              if (masked) {
                const int key = blk * 16 + h * 8 + 2 * t;
                const bool there_a = (valid >> key) & 1u, there_b = (valid >> (key + 1)) & 1u;
                const bool fine_a = q4_finite(q4_pair(pa)), fine_b = q4_finite(q4_pair(pb));
                if ((there_a && !fine_a) || (there_b && !fine_b)) ctl.bad = 1;
                if (!there_a || !fine_a) pa = 0u;
                if (!there_b || !fine_b) pb = 0u;
              }
              sp[h] = as_half2(__byte_perm(pa, pb, 0x5410));
              mp[h] = as_half2(__byte_perm(pa, pb, 0x7632));
            }
            constexpr int kWords = D / 64;  // of a token that this lane has
#pragma unroll
            for (int x = 0; x < kWords; ++x) {
              uint32_t lo[2], hi[2];  // the even and the odd dimensions of two tokens
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const char *at = v0 + h * 8 * kRow + (g * kWords + x) * 4;
                const uint32_t xa = *reinterpret_cast<const uint32_t *>(at);
                const uint32_t xb = *reinterpret_cast<const uint32_t *>(at + kRow);
                lo[h] = __byte_perm(xa, xb, 0x5410);
                hi[h] = __byte_perm(xa, xb, 0x7632);
              }
#pragma unroll
              for (int s = 0; s < 4; ++s) {
                auto value = [&](uint32_t codes, int h) {
                  const __half2 n =
                      s & 1 ? __hsub2(as_half2((codes & 0x00F000F0u) | 0x54005400u), as_half2(0x54005400u))
                            : __hsub2(as_half2((codes & 0x000F000Fu) | 0x64006400u), as_half2(0x64006400u));
                  return as_word(__hfma2(n, sp[h], mp[h]));
                };
                const uint32_t a0 = value(lo[0], 0), a1 = value(hi[0], 0), a2 = value(lo[1], 1),
                               a3 = value(hi[1], 1);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma16(o[nt][x * 4 + s], a0, a1, a2, a3, w[blk][nt][0], w[blk][nt][1]);
                if (s & 1) {
                  lo[0] >>= 8, lo[1] >>= 8, hi[0] >>= 8, hi[1] >>= 8;
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&ctl.empty[st]);
      }

      // the unit's end: the warps' results meet, half of the dimensions at a time
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int s = 4; s <= 16; s <<= 1) l[nt][e] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][e], s);
          if (g == 0) {
            ml_s[warp][0][nt * 8 + 2 * t + e] = m[nt][e];
            ml_s[warp][1][nt * 8 + 2 * t + e] = l[nt][e];
          }
        }
      float *meet = reinterpret_cast<float *>(smem4 + L::kMeet);
      const bool whole = u.whole();
      float *slot = p.part + piece_slot(u, line.worker) * slot_floats(p.rows, D);
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        if ((g >> 2) == half) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int j = 0; j < kOuts; j += 2) {
                // dimensions 2j .. 2j + 3 of this lane's D / 8
                float *to = meet + warp * L::kMeetFloats + (nt * 8 + 2 * t + e) * (D / 2) + (g & 3) * (D / 8) + 2 * j;
                *reinterpret_cast<float4 *>(to) =
                    make_float4(o[nt][j][e], o[nt][j][2 + e], o[nt][j + 1][e], o[nt][j + 1][2 + e]);
              }
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        for (int i = tid; i < R * (D / 8); i += 32 * kQ4Warps) {
          const int row = i / (D / 8), x = i % (D / 8) * 4, d = half * (D / 2) + x;
          if (row >= live) continue;
          float M = -INFINITY, sum = 0.f;
#pragma unroll
          for (int w = 0; w < kQ4Warps; ++w) M = fmaxf(M, ml_s[w][0][row]);
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kQ4Warps; ++w) {
            // a part is empty where its sum is zero: one of NaN scores has m -infinity too
            if (ml_s[w][1][row] == 0.f) continue;
            const float f = fast_exp2(ml_s[w][0][row] - M);
            const float4 part = *reinterpret_cast<const float4 *>(meet + w * L::kMeetFloats + row * (D / 2) + x);
            sum += f * ml_s[w][1][row];
            v.x += f * part.x;
            v.y += f * part.y;
            v.z += f * part.z;
            v.w += f * part.w;
          }
          if (*reinterpret_cast<volatile int *>(&ctl.bad))
            v = nonfinite_values_q4<D>(p, u, (u.r0 + row) / p.G, d, v);
          if (whole) {
            const long long at = out_row(p, u.b, u.h, u.r0 + row);
            const float n = sum == 0.f ? 0.f : 1.f / sum;
            store4(static_cast<TE *>(p.out) + at * D + d, make_float4(v.x * n, v.y * n, v.z * n, v.w * n));
            if (d == 0 && p.lse) p.lse[at] = row_lse(M, sum);
          } else {
            store4(slot + slot_stats(p.rows) + static_cast<size_t>(row) * D + d, v);
            if (d == 0) {
              slot[row] = M;
              slot[p.rows + row] = sum;
            }
          }
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
      }
    } while (u.next(p, line));
  }
  __syncthreads();
  if (ctl.dead) void_run<E, D, kQ4Threads>(p, line);
}

namespace {

template <class E, int D, int NT>
cudaError_t start4(const AttnParams &p, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr int smem = Rows4<D, NT>::kSmem;
  return launch_large(rows4_kernel<E, D, NT>, done, smem, p.workers, kQ4Threads, smem, stream, p);
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
