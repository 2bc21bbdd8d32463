// Attention over a paged cache of 4-bit rows (q4.cuh): head_dim 64 or 128, queries and
// outputs of 16 bits, 4 or 8 rows of queries per unit (new tokens times the group's heads).
//
// A warp is a worker: it has units of its own, copies 32 keys and their values at a time
// into a ring of its own, two ahead, and writes its units' outputs, without a barrier.
//
// Scores: the keys are the rows of the matrix instruction and the queries its columns.  A
// code n, masked out of its word and taken as float16, is the subnormal n 2^-24 (16 n
// 2^-24 for the odd nibbles, whose queries are divided by 16): the products are exact, and
// cost a mask each.  Each of the four groups of a row has sums of its own; a key's score is
//   sum over groups g of s_g (q . n)_g + m_g (sum of q)_g
// with the scales applied to the sums in float32 and the minima as one more step of
// the instruction, against the queries' sums in two float16 terms.  So scores are as
// exact as those of rows in float16 without any value being made.  Queries enter as
// float16, each row scaled by a power of two to 2^9 at most: exact but for what lies
// 2^-24 below a row's largest.  Four rows leave half of the eight columns free: those take
// another group's codes, with zeros against the first's.
//
// Outputs: the values are the rows, the keys the inner dimension, the codes the same
// subnormals.  The scales go into the weights, one product of float16 per key, row and
// group instead of one per key and value; sums of the weights times the minima are two
// more columns.  Weights are float16 as in the tensor-memory kernels: lifted, so that
// those rounded to zero are below 2^-31 of the row's largest; the product with a scale
// rounds once more (half a step of 2^-11, against quantisation by half a step of 1/15 of
// the spread).  Powers of two keep both in float16's range whatever the scales are
// (bring_near_one): a product is lost below 2^-24 of the row's largest weight times the
// group's usual scale.  The weights of 8 keys and 8 rows cross from the scores' layout to the
// products' by one transposing move.
//
// Bound by instructions and the latencies between them: 690 for 32 keys and values, issued
// in every second cycle by the three warps a scheduler has registers for (sixteen warps an
// SM instead of twelve, with fewer registers: 179 us).  256 sequences of 1 to 4096 tokens,
// one token each, 32/8 heads of 128: 158 us, 4.27 TB/s; the copies alone take 112.
#include <algorithm>

#include "q4_copies.cuh"

namespace sv {

namespace {

constexpr int kQ4Tile = kQ4Keys;  // of a tile
constexpr int kSms4 = 152;
// Weights reach 2^(kLift4 + kSlack) = 2^14, and times scales below 2 stay in float16.
constexpr float kLift4 = 6.f;

// R: rows of a unit, 4 or 8.
template <int D, int R>
struct Rows4 {
  static constexpr int kRow = q4_row_bytes(D);
  // Four rows leave half of the products' columns free, which take another group.
  static constexpr bool kQuad = R == 4;
  static constexpr int kWarps = 4;                     // of a CTA
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kCtas = 3;                      // of an SM (four: 179 us for 157)
  static constexpr int kStage = 2 * kQ4Tile * kRow;    // keys, then values
  static constexpr int kSteps = D / 16;                // of the scores' products
  // of the queries: two operands a step, two for the sums, the factors; two steps a piece
  static constexpr int kQPieces = kSteps / 2 + 1;
  static constexpr int kQBytes = kQPieces * 32 * 16;
  // usual_downs of the unit; bring_near_one of the tile's keys
  static constexpr int kDowns = 2 * kStage + kQBytes;
  static constexpr int kBy = kDowns + 16;
  static constexpr int kWarp = kBy + 4 * kQ4Tile;
  static constexpr int kSmem = kWarps * kWarp;
  static_assert(kCtas * (kSmem + 2048) <= 227 * 1024, "shared memory of an SM");
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
// 8x8 matrices of 16-bit halves; with "memory": the ring's contents change under them.
__device__ __forceinline__ void matrices4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void matrices4_turned(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void matrices2(uint32_t (&r)[2], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at) : "memory");
}
__device__ __forceinline__ void matrices2_turned(uint32_t (&r)[2], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
               : "=r"(r[0]), "=r"(r[1])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t as_word(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }
__device__ __forceinline__ float scale_at(const char *p) { return __half2float(*reinterpret_cast<const __half *>(p)); }
constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;  // nibbles of two halves

// The products of weights and scales are float16, so a key's scales are brought near one, and
// its weight times the same power of two takes their place in the row's running maximum:
// neither small scales nor a key of large ones costs the other keys' weights their bits.
// Tiles of scales within [1/128, 2) stay as they are (others take 180 us where those take 161:
// one token at B = 256, 1 to 4096 tokens).

// Not zero where a scale lies outside of [1/128, 2): its exponent field outside of 8 to 15.
__device__ __forceinline__ uint32_t scale_far(uint32_t pair) { return (pair ^ 0x2000u) & 0x6000u; }
__device__ __forceinline__ bool scales_far(uint4 s) {
  return (scale_far(s.x) | scale_far(s.y) | scale_far(s.z) | scale_far(s.w)) != 0u;
}
// Exponent field of a scale; -1: zero, or not finite.
__device__ __forceinline__ int scale_field(uint32_t pair) {
  const uint32_t x = pair & 0x7FFFu;
  return x != 0u && x < 0x7C00u ? static_cast<int>(x >> 10) : -1;
}
// Groups whose scales are usually smaller than another group's: by how many powers of two, a
// byte a group, at most 7, so that keys whose groups are alike are not brought further apart
// than the groups of tiles that stay as they are.  By a whole warp, from a tile's keys.
__device__ __forceinline__ uint32_t usual_downs(uint4 s) {
  const uint32_t w[4] = {s.x, s.y, s.z, s.w};
  int mean[4], top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int field = scale_field(w[j]);
    const uint32_t sum = __reduce_add_sync(0xFFFFFFFFu, field < 0 ? 0u : 0x10000u + field);
    const int n = sum >> 16;
    mean[j] = n ? (static_cast<int>(sum & 0xFFFFu) + n / 2) / n : -1;
    top = max(top, mean[j]);
  }
  uint32_t downs = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    downs |= static_cast<uint32_t>(mean[j] < 0 ? 0 : min(top - mean[j], 7)) << (8 * j);
  return downs;
}
__device__ __forceinline__ int down_exponent(uint32_t downs, int group) { return downs >> (8 * group) & 255; }
__device__ __forceinline__ float down_of(uint32_t downs, int group) {
  return __int_as_float((127 - down_exponent(downs, group)) << 23);
}
// Brings the largest of a key's scales, times 2^downs, into [1, 2), and its minima with them;
// returns the power of two that its weight takes instead.  Small scales are raised no further
// than float16 holds the minima.
__device__ __forceinline__ int bring_near_one(uint4 &s, uint32_t downs) {
  uint32_t *w = reinterpret_cast<uint32_t *>(&s);
  int high = -1, low = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int field = scale_field(w[j]), minimum = w[j] >> 26 & 31;
    if (field >= 0) high = max(high, field + down_exponent(downs, j));
    if (minimum < 31) low = max(low, minimum);
  }
  const int by = high < 0 ? 0 : max(high - 15, low - 30);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = q4_pair(w[j]);
    w[j] = F16::pack(x.x * __int_as_float((127 + down_exponent(downs, j) - by) << 23),
                     x.y * __int_as_float((127 - by) << 23));
  }
  return by;
}

// A lane's operands of the scores' products, of the unit's queries as eight columns
// (four with kQuad), into pieces of 16 bytes [step / 2][lane]:
//   kQuad, D 128, step 4 pr + i: nibble i of group 2 pr in columns 0..3, of group 2 pr + 1
//     in columns 4..7, each with zeros for the other's keys' codes
//   kQuad, D 64, step 2 pc + i: nibbles 2i, 2i + 1 of words 4 pc + t: columns 0..3 of the
//     first two (group 2 pc), 4..7 of the others
//   D 128, step 2 j + i: nibbles 2i, 2i + 1 of group j; D 64, step j: group j
// then the sums of each group in two float16 terms, against the codes' (scale, minimum)
// pairs, and the factors of this lane's two rows of scores.
template <class E, int D, bool kQuad>
__device__ __forceinline__ void prepare_queries(const AttnParams &p, const UnitWalk &u, int lane, uint4 *to) {
  using TE = typename E::T;
  constexpr int kN = D / 16;         // values of each group that this lane has
  constexpr bool kPieces = D == 128 || kQuad;  // in pieces of eight neighbours
  constexpr int kParts = kPieces ? D / 32 : 4, kEach = kPieces ? 8 : kN;
  const int g = lane >> 2, t = lane & 3, live = u.live_rows(p), row = kQuad ? g & 3 : g;
  const int r = u.r0 + min(row, live - 1), n = r / p.G;
  const char *q = p.q + u.b * p.q_seq + n * p.q_token + (u.h * p.G + r - n * p.G) * p.q_head;
  uint32_t v[kParts][kEach / 2];
#pragma unroll
  for (int j = 0; j < kParts; ++j) {
    const TE *from = reinterpret_cast<const TE *>(q) + j * (D / kParts) + t * kEach;
    if constexpr (kEach == 8) {
      const uint4 y = *reinterpret_cast<const uint4 *>(from);
      v[j][0] = y.x, v[j][1] = y.y, v[j][2] = y.z, v[j][3] = y.w;
    } else {
      const uint2 y = *reinterpret_cast<const uint2 *>(from);
      v[j][0] = y.x, v[j][1] = y.y;
    }
  }
  float x[kParts][kEach];
  float top = 0.f;
  bool odd = false;
#pragma unroll
  for (int j = 0; j < kParts; ++j)
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
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
  // a query that is not finite makes its row's scores NaN, those that the mask leaves
  const float factor = odd ? __int_as_float(0x7FC00000)
                           : p.scale_log2 * __int_as_float((127 - exponent) << 23);
  float sum[kParts];
#pragma unroll
  for (int j = 0; j < kParts; ++j) {
    sum[j] = 0.f;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      // as the products see it
      x[j][e] = odd ? 0.f : __half2float(__float2half_rn(x[j][e] * up));
      sum[j] += x[j][e];
    }
    sum[j] += __shfl_xor_sync(0xFFFFFFFFu, sum[j], 1);
    if (kEach * 4 == D / 4) sum[j] += __shfl_xor_sync(0xFFFFFFFFu, sum[j], 2);
  }
  // the sum of group t
  float mine = 0.f;
  if constexpr (kEach * 4 == D / 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t == j) mine = sum[j];
  } else {
    // a piece is two groups: lanes 0, 1 of four have the first, 2, 3 the second
    const int from = (lane & ~3) | (2 * (t & 1));
    const float s0 = __shfl_sync(0xFFFFFFFFu, sum[0], from), s1 = __shfl_sync(0xFFFFFFFFu, sum[1], from);
    mine = t >> 1 ? s1 : s0;
  }
  if (kQuad && g >= 4) mine = 0.f;
  auto pair = [&](int j, int i) {  // nibble i of this lane's word j
    const float f = i & 1 ? 0.0625f : 1.f;
    return F16::pack(x[j][2 * i] * f, x[j][2 * i + 1] * f);
  };
  uint32_t b[kN * 2];
  if constexpr (kQuad && D == 128) {
#pragma unroll
    for (int pr = 0; pr < 2; ++pr)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        b[(pr * 4 + i) * 2] = g < 4 ? pair(2 * pr, i) : 0u;
        b[(pr * 4 + i) * 2 + 1] = g < 4 ? 0u : pair(2 * pr + 1, i);
      }
  } else if constexpr (kQuad) {
    const bool here = (g >> 2) == (t >> 1);
#pragma unroll
    for (int pc = 0; pc < 2; ++pc)
#pragma unroll
      for (int i = 0; i < 4; ++i) b[pc * 4 + i] = here ? pair(pc, i) : 0u;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < kEach / 2; ++i) b[j * (kEach / 2) + i] = pair(j, i);
  }
#pragma unroll
  for (int i = 0; i < kN / 2; ++i) to[i * 32] = make_uint4(b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3]);
  const __half hi = __float2half_rn(mine), lo = __float2half_rn(mine - __half2float(hi));
  const int row0 = kQuad ? 2 * (t & 1) : 2 * t;
  to[kN / 2 * 32] = make_uint4(static_cast<uint32_t>(__half_as_ushort(hi)) << 16,
                               static_cast<uint32_t>(__half_as_ushort(lo)) << 16,
                               __float_as_uint(__shfl_sync(0xFFFFFFFFu, factor, row0 * 4)),
                               __float_as_uint(__shfl_sync(0xFFFFFFFFu, factor, (row0 + 1) * 4)));
}

}  // namespace

template <class E, int D, int R>
__global__ void __launch_bounds__(Rows4<D, R>::kThreads, Rows4<D, R>::kCtas)
    rows4_kernel(const __grid_constant__ AttnParams p) {
  using L = Rows4<D, R>;
  using TE = typename E::T;
  constexpr int kRow = L::kRow;
  constexpr bool kQuad = L::kQuad, kPieces = D == 128 || kQuad;
  extern __shared__ __align__(128) char smem4[];
  __shared__ RunScratch<L::kThreads, L::kWarps> runs;
  __shared__ Line lines_s[L::kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  {
    Line lines[L::kWarps];
    // consecutive workers on different CTAs
    find_runs(p, runs, blockIdx.x, gridDim.x, lines);
#pragma unroll
    for (int w = 0; w < L::kWarps; ++w)
      if (tid == w * 32) lines_s[w] = lines[w];
  }
  __syncwarp();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Line &line = lines_s[warp];
  UnitWalk u;
  bool busy = u.start(p, line);
  if (lane == 0) write_join(p, line, busy ? &u : nullptr);

  const int g = lane >> 2, t = lane & 3;
  constexpr int kOuts = D / 16;    // 16 dimensions each of the outputs
  constexpr int kKeys = kQuad ? 1 : 2;  // of 16, that this lane weighs
  auto key_of = [&](int h) { return kQuad ? (t >> 1) * 8 + g : h * 8 + g; };
  auto row_of = [&](int e) { return kQuad ? 2 * (t & 1) + e : 2 * t + e; };
  // where this lane's row of a matrix of codes begins: keys 0..7 and 8..15 of one piece of
  // 16 bytes, then of the next
  const int matrix = ((lane & 7) + ((lane >> 3) & 1) * 8) * kRow + (lane >> 4) * 16;
  char *ring = smem4 + warp * L::kWarp;
  const uint32_t ring_at = smem_u32(ring);
  uint4 *queries = reinterpret_cast<uint4 *>(ring + 2 * L::kStage) + lane;
  Q4Copies<kRow> copies(p, lane);
  uint32_t asked = 0, tiles = 0;  // tiles copied, and weighed
  uint32_t there[2] = {0u, 0u};   // which of a tile's keys were copied
  auto ask = [&](int i) {
    const uint32_t st = asked++ & 1u;
    const uint32_t word = copies.ask(p, u, key_tile(u.k, i) * kQ4Tile, ring_at + st * L::kStage, lane);
    there[0] = st ? there[0] : word;
    there[1] = st ? word : there[1];
  };

  if (busy) copies.begin(p, u, key_tile(u.k, u.i0) * kQ4Tile, lane);
  uint32_t *unit_downs = reinterpret_cast<uint32_t *>(ring + L::kDowns);
  while (busy) {
      if (lane == 0) *unit_downs = 0u;
      prepare_queries<E, D, kQuad>(p, u, lane, queries);
    __syncwarp();
    uint32_t qs[2];
    float c[2];
    const int live = u.live_rows(p);
    {
      const uint4 x = queries[(L::kSteps / 2) * 32];
      qs[0] = x.x;
      qs[1] = x.y;
      c[0] = __uint_as_float(x.z);
      c[1] = __uint_as_float(x.w);
    }
    float m[2], l[2], o[kOuts][4], om[4];
    {
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
      om[0] = om[1] = om[2] = om[3] = 0.f;
#pragma unroll
      for (int i = 0; i < kOuts; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
    bool bad = false;

    // two tiles are on their way while one is weighed
    for (int i = u.i0 - 2; i < u.i1; ++i) {
      uint32_t valid = 0u;
      const uint32_t st = tiles & 1u;
      if (i >= u.i0) {
        copy_wait<1>();
        __syncwarp();
        ++tiles;
        valid = st ? there[1] : there[0];
      }
      if (valid != 0u) {
      const int at0 = key_tile(u.k, i) * kQ4Tile;
      char *k_s = ring + st * L::kStage, *v_s = k_s + kQ4Tile * kRow;
      const uint32_t k_at = ring_at + st * L::kStage, v_at = k_at + kQ4Tile * kRow;
      // this lane's key: its values' scales
      uint4 *scales = reinterpret_cast<uint4 *>(v_s + lane * kRow + D / 2);
      uint4 s = *scales;
      const bool masked = valid != 0xFFFFFFFFu || !all_seen(p, u.k, at0, kQ4Tile);
      bool far = scales_far(s);
      if (masked) {
        // rows that were not copied stand for zeros, and so do groups that are not
        // finite, which nonfinite_values_q4 adds
        uint32_t *w = reinterpret_cast<uint32_t *>(&s);
        const bool copied = (valid >> lane) & 1u;
        uint32_t apart = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (!copied || !q4_finite(w[j])) {
            bad |= copied;
            w[j] = 0u;
          } else {
            apart |= scale_far(w[j]);
          }
        far = apart != 0u;
      }
      uint32_t downs = *unit_downs;
      const bool moved = __any_sync(0xFFFFFFFFu, far || downs != 0u);
      if (moved) {
        // (where no row has a maximum the outputs so far are zeros, whatever they were times)
        if (__all_sync(0xFFFFFFFFu, m[0] == -INFINITY && m[1] == -INFINITY)) {
          downs = usual_downs(s);
          *unit_downs = downs;  // the same in every lane
        }
        reinterpret_cast<int *>(ring + L::kBy)[lane] = bring_near_one(s, downs);
      }
      if (masked || moved) {
        *scales = s;
        __syncwarp();
      }
      // (once in the code: unrolled, its instructions do not stay in the cache, 12 % slower)
#pragma unroll 1
      for (int blk = 0; blk < 2; ++blk) {
        // ------------------------------------------------------------- scores
        float y[2 * kKeys];
        const char *r0 = k_s + (blk * 16 + g) * kRow, *r1 = r0 + 8 * kRow;
        uint32_t pairs[2];
        matrices2(pairs, k_at + (blk * 16 + (lane & 15)) * kRow + D / 2);
        if constexpr (kQuad) {
          float a[2][4], am[4];
#pragma unroll
          for (int pr = 0; pr < 2; ++pr) {
            uint32_t r[4];
            if constexpr (D == 128) {
              matrices4(r, k_at + matrix + blk * 16 * kRow + pr * 32);
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                const uint4 q = queries[(pr * 2 + i / 2) * 32];
                if (i == 0) {
                  mma16_first(a[pr], r[0] & kLow, r[1] & kLow, r[2] & kLow, r[3] & kLow, q.x, q.y);
                } else {
                  mma16(a[pr], r[0] & kLow, r[1] & kLow, r[2] & kLow, r[3] & kLow, q.x, q.y);
                }
                mma16(a[pr], r[0] & kHigh, r[1] & kHigh, r[2] & kHigh, r[3] & kHigh, q.z, q.w);
#pragma unroll
                for (int x = 0; x < 4; ++x) r[x] >>= 8;
              }
            } else {
              // two pieces of 16 bytes: this one's keys 0..7 and 8..15
              const uint4 q = queries[pr * 32];
              uint32_t r2[2];
              matrices2(r2, k_at + (blk * 16 + (lane & 15)) * kRow + pr * 16);
              mma16_first(a[pr], r2[0] & kLow, r2[1] & kLow, r2[0] & kHigh, r2[1] & kHigh, q.x, q.y);
              r2[0] >>= 8, r2[1] >>= 8;
              mma16(a[pr], r2[0] & kLow, r2[1] & kLow, r2[0] & kHigh, r2[1] & kHigh, q.z, q.w);
            }
          }
          mma16_first(am, pairs[0], pairs[1], pairs[0], pairs[1], qs[0], qs[1]);
          // columns 0..3 are groups 0 and 2, 4..7 the same rows' groups 1 and 3
          const char *f0 = r0 + D / 2 + (t >> 1) * 4, *f1 = f0 + 8 * kRow;
          const float s00 = scale_at(f0), s02 = scale_at(f0 + 8), s10 = scale_at(f1), s12 = scale_at(f1 + 8);
          float z[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            z[e] = fmaf(fmaf(e < 2 ? s02 : s12, a[1][e], (e < 2 ? s00 : s10) * a[0][e]), 16777216.f, am[e]);
          // lanes 0, 1 of four go on with the first eight keys, 2, 3 with the second
          const bool second = t >= 2;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float other = __shfl_xor_sync(0xFFFFFFFFu, second ? z[e] : z[2 + e], 2);
            y[e] = ((second ? z[2 + e] : z[e]) + other) * c[e];
          }
        } else {
          float a[4][4], am[4];
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            if constexpr (D == 128) {
              uint32_t r[4];
              matrices4(r, k_at + matrix + blk * 16 * kRow + j * 16);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t x0 = r[2 * x], x1 = r[2 * x + 1], z0 = x0 >> 8, z1 = x1 >> 8;
                const uint4 q = queries[(j + x) * 32];
                mma16_first(a[j + x], x0 & kLow, x1 & kLow, x0 & kHigh, x1 & kHigh, q.x, q.y);
                mma16(a[j + x], z0 & kLow, z1 & kLow, z0 & kHigh, z1 & kHigh, q.z, q.w);
              }
            } else {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int at = (j + x) * 8 + (t >> 1) * 4, shift = (t & 1) * 8;
                const uint32_t x0 = word_at(r0 + at) >> shift, x1 = word_at(r1 + at) >> shift;
                const uint4 q = queries[(j / 2) * 32];
                mma16_first(a[j + x], x0 & kLow, x1 & kLow, x0 & kHigh, x1 & kHigh, x ? q.z : q.x,
                            x ? q.w : q.y);
              }
            }
          }
          const uint4 s0 = *reinterpret_cast<const uint4 *>(r0 + D / 2);
          const uint4 s1 = *reinterpret_cast<const uint4 *>(r1 + D / 2);
          const float f0[4] = {__low2float(as_half2(s0.x)), __low2float(as_half2(s0.y)),
                               __low2float(as_half2(s0.z)), __low2float(as_half2(s0.w))};
          const float f1[4] = {__low2float(as_half2(s1.x)), __low2float(as_half2(s1.y)),
                               __low2float(as_half2(s1.z)), __low2float(as_half2(s1.w))};
          mma16_first(am, pairs[0], pairs[1], pairs[0], pairs[1], qs[0], qs[1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float *f = e < 2 ? f0 : f1;
            const float z = fmaf(f[3], a[3][e],
                                 fmaf(f[2], a[2][e], fmaf(f[1], a[1][e], f[0] * a[0][e])));
            y[e] = fmaf(z, 16777216.f, am[e]) * c[e & 1];
          }
        }
        if (masked) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int n = (u.r0 + min(row_of(e), live - 1)) / p.G;
#pragma unroll
              for (int h = 0; h < kKeys; ++h) {
                const int key = blk * 16 + key_of(h);
                if (!((valid >> key) & 1u) || !sees(p, u.k, u.b, n, at0 + key)) y[2 * h + e] = -INFINITY;
              }
            }
        }
        // ------------------------------------------------------------ weights
        // the product with a key's scales takes its weight times 2^by; their sum takes it as it is
        float back[kKeys];
#pragma unroll
        for (int h = 0; h < kKeys; ++h) {
          back[h] = 1.f;
          if (moved) {
            const int up = reinterpret_cast<int *>(ring + L::kBy)[blk * 16 + key_of(h)];
            y[2 * h] += static_cast<float>(up);
            y[2 * h + 1] += static_cast<float>(up);
            back[h] = __int_as_float((127 - up) << 23);
          }
        }
        auto top_of = [&](int e) { return kQuad ? y[e] : fmaxf(y[e], y[2 * (kKeys - 1) + e]); };
        bool up = false;
#pragma unroll
          for (int e = 0; e < 2; ++e) up |= top_of(e) - kLift4 > m[e] + kSlack;
        if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = top_of(e);
#pragma unroll
              for (int x = kQuad ? 2 : 4; x <= 16; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
              top -= kLift4;
              const float to = top > m[e] + kSlack ? top : m[e];
              const float f = m[e] == -INFINITY ? 0.f : fast_exp2(m[e] - to);
              m[e] = to;
              l[e] *= f;
              // (with kQuad columns 4..7 are not looked at, or hold the same rows)
              om[e] *= f;
              om[2 + e] *= f;
#pragma unroll
              for (int j = 0; j < kOuts; ++j) {
                o[j][e] *= f;
                o[j][2 + e] *= f;
              }
            }
        }
        uint32_t w[2];
        // a row that has seen nothing yet keeps weights of zero
        const float u0 = m[0] == -INFINITY ? 0.f : m[0], u1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
        for (int h = 0; h < kKeys; ++h) {
          const float p0 = fast_exp2(y[2 * h] - u0), p1 = fast_exp2(y[2 * h + 1] - u1);
          l[0] = fmaf(p0, back[h], l[0]);
          l[1] = fmaf(p1, back[h], l[1]);
          w[h] = transposed(F16::pack(p0, p1));
        }
        if constexpr (kQuad) {
          // columns 0..3 have the first eight keys' weights here, 4..7 the same rows' of the
          // second
          const uint32_t own = w[0], other = __shfl_xor_sync(0xFFFFFFFFu, own, 16);
          w[0] = g < 4 ? own : other;
          w[1] = g < 4 ? other : own;
        }
        // ------------------------------------------------------------ outputs
        // tokens 2t, 2t + 1 of the first eight keys (h = 0) and of the second
        const char *v0 = v_s + (blk * 16 + 2 * t) * kRow;
        uint32_t low[2];  // row 2j + 1: minima of group j
        matrices2_turned(low, v_at + (blk * 16 + (lane & 15)) * kRow + D / 2);
        mma16(om, low[0], 0u, low[1], 0u, w[0], w[1]);
        if constexpr (kPieces) {
          // scales of this column's group: of all four, or (D 64) of two pieces'
          uint32_t sp[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const char *va = v0 + h * 8 * kRow + D / 2, *vb = va + kRow;
            if constexpr (D == 128) {
              const uint4 pa = *reinterpret_cast<const uint4 *>(va), pb = *reinterpret_cast<const uint4 *>(vb);
              sp[h][0] = __byte_perm(pa.x, pb.x, 0x5410);
              sp[h][1] = __byte_perm(pa.y, pb.y, 0x5410);
              sp[h][2] = __byte_perm(pa.z, pb.z, 0x5410);
              sp[h][3] = __byte_perm(pa.w, pb.w, 0x5410);
            } else {
              const int x = (g >> 2) * 4;
              sp[h][0] = __byte_perm(word_at(va + x), word_at(vb + x), 0x5410);
              sp[h][1] = __byte_perm(word_at(va + x + 8), word_at(vb + x + 8), 0x5410);
            }
          }
#pragma unroll
          for (int j = 0; j < D / 32; j += 2) {
            uint32_t r[4];
            matrices4_turned(r, v_at + matrix + blk * 16 * kRow + j * 16);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t x0 = r[2 * x], x1 = r[2 * x + 1], z0 = x0 >> 8, z1 = x1 >> 8;
              const uint32_t b0 = as_word(__hmul2(as_half2(w[0]), as_half2(sp[0][j + x])));
              const uint32_t b1 = as_word(__hmul2(as_half2(w[1]), as_half2(sp[1][j + x])));
              mma16(o[2 * (j + x)], x0 & kLow, x0 & kHigh, x1 & kLow, x1 & kHigh, b0, b1);
              mma16(o[2 * (j + x) + 1], z0 & kLow, z0 & kHigh, z1 & kLow, z1 & kHigh, b0, b1);
            }
          }
        } else {
          // a group is two words: this lane's nibble of both dimensions
          const uint32_t nibble = g & 1 ? kHigh : kLow;
          const int byte = (g >> 1) & 1;
          // (the halves' upper bytes are whatever byte 0 is, and masked out)
          const uint32_t sel_even = byte | (4 + byte) << 8, sel_odd = (2 + byte) | (6 + byte) << 8;
          uint4 pa[2], pb[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            pa[h] = *reinterpret_cast<const uint4 *>(v0 + h * 8 * kRow + D / 2);
            pb[h] = *reinterpret_cast<const uint4 *>(v0 + (h * 8 + 1) * kRow + D / 2);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t a[4], sp[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const char *at = v0 + h * 8 * kRow + j * 8 + (g >> 2) * 4;
              const uint32_t xa = word_at(at), xb = word_at(at + kRow);
              a[2 * h] = __byte_perm(xa, xb, sel_even) & nibble;
              a[2 * h + 1] = __byte_perm(xa, xb, sel_odd) & nibble;
              sp[h] = __byte_perm(reinterpret_cast<const uint32_t *>(&pa[h])[j],
                                  reinterpret_cast<const uint32_t *>(&pb[h])[j], 0x5410);
            }
              mma16(o[j], a[0], a[1], a[2], a[3], as_word(__hmul2(as_half2(w[0]), as_half2(sp[0]))),
                    as_word(__hmul2(as_half2(w[1]), as_half2(sp[1]))));
          }
        }
      }
      }
      __syncwarp();
      if (i + 2 < u.i1) ask(i + 2);
      copy_commit();
    }
    // the next unit's pages and queries are on their way while this one ends
    const UnitWalk v = u;
    busy = u.next(p, line);
    if (busy) {
      copies.begin(p, u, key_tile(u.k, u.i0) * kQ4Tile, lane);
      const int r = u.r0 + min(lane / 2, u.live_rows(p) - 1), n = r / p.G;
      const char *q = p.q + u.b * p.q_seq + n * p.q_token + (u.h * p.G + r - n * p.G) * p.q_head;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(q + (lane & 1) * D) : "memory");
    }

    // the unit's end.  A lane has 16 bytes of float32 outputs at a time, of row
    // row_of(e): dimensions d0, d0 + 1, d1, d1 + 1
    const bool whole = v.whole();
    bad = __any_sync(0xFFFFFFFFu, bad);
    const uint32_t downs = *unit_downs;
    __syncwarp();
    float *slot = p.part + piece_slot(v, line.worker) * slot_floats(p.rows, D);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[e];
#pragma unroll
        for (int x = kQuad ? 2 : 4; x <= 16; x <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
        const int row = row_of(e);
        // with kQuad half of the columns are another group's, or not looked at
        const bool mine = row < live && (!kQuad || (t >> 1) == (D == 128 ? 0 : g >> 2));
        const long long at = mine ? out_row(p, v.b, v.h, v.r0 + row) : 0;
        const float n = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
        uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<TE *>(p.out) + at * D);
        float *to = slot + slot_stats(p.rows) + static_cast<size_t>(row) * D;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          float4 y;
          int d0, d1;
          if constexpr (kPieces) {
            // codes 2i (+ 1 in odd g) of a word: neighbours swap, so that each has four
            // dimensions of it
            const int group = D == 128 ? j : 2 * j + (g >> 2);
            const float lo = __shfl_sync(0xFFFFFFFFu, om[e], (2 * group + 1) * 4 + t);
            const float even = 16777216.f * down_of(downs, group), odds = even * 0.0625f;
            const float x0 = fmaf(o[2 * j][e], even, lo), x1 = fmaf(o[2 * j][2 + e], odds, lo);
            const float x2 = fmaf(o[2 * j + 1][e], even, lo), x3 = fmaf(o[2 * j + 1][2 + e], odds, lo);
            const bool odd = g & 1;
            const float z0 = __shfl_xor_sync(0xFFFFFFFFu, odd ? x0 : x2, 4);
            const float z1 = __shfl_xor_sync(0xFFFFFFFFu, odd ? x1 : x3, 4);
            y = odd ? make_float4(z0, x2, z1, x3) : make_float4(x0, z0, x1, z1);
            d0 = 32 * j + 4 * g;
            d1 = d0 + 2;
          } else {
            const float lo = __shfl_sync(0xFFFFFFFFu, om[e], (4 * j + 1) * 4 + t);
            const float hi = __shfl_sync(0xFFFFFFFFu, om[e], (4 * j + 3) * 4 + t);
            const float f = g & 1 ? 1048576.f : 16777216.f;
            const float f0 = f * down_of(downs, 2 * j), f1 = f * down_of(downs, 2 * j + 1);
            y = make_float4(fmaf(o[2 * j][e], f0, lo), fmaf(o[2 * j][2 + e], f0, lo),
                            fmaf(o[2 * j + 1][e], f1, hi), fmaf(o[2 * j + 1][2 + e], f1, hi));
            d0 = 32 * j + 2 * g;
            d1 = d0 + 16;
          }
          if (!mine) continue;
          if (bad) {
            const int token = (v.r0 + row) / p.G;
            const float2 z0 = nonfinite_values_q4<D, kQ4Tile>(p, v, token, d0), z1 = nonfinite_values_q4<D, kQ4Tile>(p, v, token, d1);
            y.x += z0.x, y.y += z0.y, y.z += z1.x, y.w += z1.y;
          }
          const uint2 packed = make_uint2(E::pack(y.x * n, y.y * n), E::pack(y.z * n, y.w * n));
          if constexpr (kPieces) {
            if (whole) {
              *reinterpret_cast<uint2 *>(out + d0 / 2) = packed;
            } else {
              *reinterpret_cast<float4 *>(to + d0) = y;
            }
          } else if (whole) {
            out[d0 / 2] = packed.x;
            out[d1 / 2] = packed.y;
          } else {
            *reinterpret_cast<float2 *>(to + d0) = make_float2(y.x, y.y);
            *reinterpret_cast<float2 *>(to + d1) = make_float2(y.z, y.w);
          }
        }
        if (mine && (g & 3) == 0 && (kQuad || g == 0)) {
          if (!whole) {
            slot[row] = m[e];
            slot[p.rows + row] = sum;
          } else if (p.lse) {
            p.lse[at] = row_lse(m[e], sum);
          }
        }
      }
  }
}

namespace {

template <class E, int D, int R>
cudaError_t start4(const AttnParams &p, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  using L = Rows4<D, R>;
  return launch_large(rows4_kernel<E, D, R>, done, L::kSmem, p.workers / L::kWarps, L::kThreads, L::kSmem,
                      stream, p);
}
template <int R>
cudaError_t start4(const AttnParams &p, int dtype, cudaStream_t stream) {
  if (dtype == SPEC_BF16)
    return p.D == 64 ? start4<Bf16, 64, R>(p, stream) : start4<Bf16, 128, R>(p, stream);
  return p.D == 64 ? start4<F16, 64, R>(p, stream) : start4<F16, 128, R>(p, stream);
}

template <int R>
AttnPlan q4_plan_of() {
  return {Rows4<128, R>::kCtas * Rows4<128, R>::kWarps * kSms4, R, 5, 2, 8};
}
// More rows go to tensor memory.  (As units of 16 rows here, whose outputs alone are 128
// registers a thread: four tokens of 32/8 heads of 128 at B = 64 119 us, 117 there, at B = 4
// 33 us and 22.  Eight rows there: 116 us, 68 here.)
bool q4_wide(int N, int G) { return N * G > 8 && G <= 128; }
AttnPlan q4_plan(int N, int G) {
  if (q4_wide(N, G))
    return N * G <= 32                  ? AttnPlan{kSms4, 32, 7, 4, 8}
           : N * G <= wide_tile_rows(G) ? AttnPlan{kSms4, wide_tile_rows(G), 7, 4, 8}
                                        : AttnPlan{kSms4, 2 * wide_tile_rows(G), 7, 8, 16};
  return N * G <= 4 ? q4_plan_of<4>() : q4_plan_of<8>();
}

}  // namespace

size_t attention_q4_workspace_bytes(int N, int G, int D) { return plan_bytes(q4_plan(N, G), D); }

cudaError_t launch_attention_q4(AttnParams &p, int dtype, void *workspace, cudaStream_t stream) {
  const bool wide = q4_wide(p.S.N, p.G);
  take_plan(p, q4_plan(p.S.N, p.G), workspace);
  // row tiles of a tree see the same keys, those of a chain end at their own
  const int tiles = (p.S.N * p.G + p.rows - 1) / p.rows;
  if (wide && p.mask && tiles <= 8) p.row_lines = tiles;
  const cudaError_t e = wide          ? launch_attention_q4_wide(p, dtype, stream)
                        : p.rows == 4 ? start4<4>(p, dtype, stream)
                                      : start4<8>(p, dtype, stream);
  if (e != cudaSuccess || p.whole) return e;
  return launch_join(p, dtype, stream);
}

}  // namespace sv
