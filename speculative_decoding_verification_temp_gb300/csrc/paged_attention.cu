// Attention over a paged cache where the tensor-memory kernels do not apply: 16
// rows of 16-bit types per unit on warp-level matrix instructions (head_dim other
// than 64 and 128, pages that are no multiple of 8 tokens, more than 128 query heads
// to one), 8 rows of float32 on the FMA pipes; and the join of the pieces of cut
// units.
//
// Each row tile reads its keys and values once.  16-bit, 256 sequences of 1 to
// 4096 tokens, one token each, 32 query heads on 8 of 128, bound by HBM: 363 us
// (5.9 TB/s) with pages of 20 tokens, where the tensor-memory kernels take 348 us
// with pages of 16 (first calls after other work); many rows are bound by the row
// tiles' re-reading: 32 trees of 60 nodes 1035 us against 115.
//
// In both kernels each of the four warps of a CTA streams its own quarter of
// each key tile through a ring of its own in shared memory (cp.async, 16 bytes
// a piece, so a row may start on any page) and keeps its own running maximum,
// sum and output in registers, so that no barrier is on the stream.  The warps'
// results meet in shared memory at the end of a unit.
//
// A weight is 2^(s c - m) with c = scale log2(e) and m the running maximum of
// s c (less a constant for float16), rounded once and then used as it is: the
// weights of all keys, the sums and the logarithm refer to the same float32 m.
#include <algorithm>

#include "paged_attention.cuh"

namespace sv {

namespace {

constexpr int kSms = 152;       // GB300
constexpr int kAttnThreads = 128;
constexpr int kAttnWarps = 4;
constexpr int kJoinThreads = 128;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
template <class E>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1);
template <>
__device__ __forceinline__ void mma<Bf16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<F16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Adds the warps' results of a unit (o_s: each warp's R x DP outputs at
// warp_floats apart; ml_s: m and l of each warp's rows) and writes the unit's
// rows, or its piece of them.  Here and in the other merges a part is empty where
// its l is zero: the maximum takes no NaN, so a part whose scores are all NaN has m
// -infinity as an empty one has, and l NaN, which reaches the row.
template <class TE, int R, int DP, int kSlice>
__device__ __forceinline__ void write_unit(const AttnParams &p, const UnitWalk &u,
                                           const float *o_s, int warp_floats,
                                           const float (*ml_s)[2][R], bool bad, int worker) {
  const int live = u.live_rows(p);
  const bool whole = u.whole();
  float *slot = p.part + piece_slot(u, worker) * slot_floats(p.rows, p.D);
  for (int i = threadIdx.x; i < R * (DP / 4); i += kAttnThreads) {
    const int row = i / (DP / 4), d = i % (DP / 4) * 4;
    if (row >= live || d >= p.D) continue;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) M = fmaxf(M, ml_s[w][0][row]);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      if (ml_s[w][1][row] == 0.f) continue;
      const float f = fast_exp2(ml_s[w][0][row] - M);
      const float4 x = *reinterpret_cast<const float4 *>(o_s + w * warp_floats + row * DP + d);
      l += f * ml_s[w][1][row];
      o.x += f * x.x;
      o.y += f * x.y;
      o.z += f * x.z;
      o.w += f * x.w;
    }
    if (bad) o = nonfinite_values<TE, kSlice>(p, u, (u.r0 + row) / p.G, d, o);
    if (whole) {
      const long long at = out_row(p, u.b, u.h, u.r0 + row);
      const float r = l == 0.f ? 0.f : 1.f / l;
      store4(static_cast<TE *>(p.out) + at * p.D + d,
             make_float4(o.x * r, o.y * r, o.z * r, o.w * r));
      if (d == 0 && p.lse) p.lse[at] = row_lse(M, l);
    } else {
      store4(slot + slot_stats(p.rows) + static_cast<size_t>(row) * p.D + d, o);
      if (d == 0) {
        slot[row] = M;
        slot[p.rows + row] = l;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// 16-bit types, 16 rows per unit
// ---------------------------------------------------------------------------

// DP: head_dim padded to 64, 128 or 256; KT: keys per warp and tile; ST: tiles
// in a warp's ring.  Shared rows of DP elements hold their 16-byte pieces
// permuted within each 128 bytes (piece ^ row mod 8), so that the eight rows of
// an 8x8 matrix load meet eight different banks.
template <int DP, int KT, int ST>
struct Rows16 {
  static constexpr int kTile = kAttnWarps * KT;
  static constexpr int kRow = DP * 2;
  static constexpr int kStage = 2 * KT * kRow;  // keys, then values
  static constexpr int kRing = ST * kStage;
  static constexpr int kSmem = 16 * kRow + kAttnWarps * kRing;
  static_assert(kRing >= 16 * DP * 4, "a warp's outputs fit its ring");
};

template <class E, int DP, int KT, int ST>
__global__ void __launch_bounds__(kAttnThreads, DP <= 128 ? 2 : 1) rows16_kernel(const __grid_constant__ AttnParams p) {
  using L = Rows16<DP, KT, ST>;
  using TE = typename E::T;
  extern __shared__ __align__(128) char smem[];
  __shared__ float ml_s[kAttnWarps][2][16];
  __shared__ uint32_t valid_s[kAttnWarps][ST];
  __shared__ int bad_s;
  __shared__ RunScratch<kAttnThreads, 1> run_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  char *q_s = smem;
  char *ring = smem + 16 * L::kRow + warp * L::kRing;
  const uint32_t q_at = smem_u32(q_s), ring_at = smem_u32(ring);
  if (p.D < DP) {
    // pieces behind head_dim are never copied to: zero for good
    for (int i = tid; i < L::kSmem / 16; i += kAttnThreads)
      reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
  }
  if (tid == 0) bad_s = 0;
  Line lines[1];
  find_runs(p, run_s, blockIdx.x, 0, lines);
  const Line &line = lines[0];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  UnitWalk u;
  const bool busy = u.start(p, line);
  if (tid == 0) write_join(p, line, busy ? &u : nullptr);
  if (!busy) return;

  // piece of a row that this lane copies, and the row of it among each batch
  constexpr int kPieces = DP / 8, kBatch = 32 / kPieces;
  const int piece = lane % kPieces, sub = lane / kPieces;
  const bool has_piece = piece * 8 < p.D;
  const float c = p.scale_log2;

  for (;;) {
    // this lane's key of the next tile to copy
    int pid = -1, in_page = 0;
    auto look_up = [&](int i) {
      pid = -1;
      const int at = key_tile(u.k, i) * L::kTile + warp * KT + lane;
      if (i < u.i1 && lane < KT && at < u.k.end) {
        const int index = at / p.C.page_size;
        in_page = at - index * p.C.page_size;
        pid = page_at(p.S, u.b, index);
      }
    };
    auto copy_tile = [&](int i) {
      if (i < u.i1) {
        const int st = (i - u.i0) % ST;
        const bool ok = page_ok(p.C, pid);
        const long long ko = ok ? pid * p.C.k_page + in_page * p.C.k_token + u.h * p.C.k_head : 0;
        const long long vo = ok ? pid * p.C.v_page + in_page * p.C.v_token + u.h * p.C.v_head : 0;
        const uint32_t valid = __ballot_sync(0xFFFFFFFFu, ok);
        if (lane == 0) valid_s[warp][st] = valid;
        const uint32_t at = ring_at + st * L::kStage;
#pragma unroll
        for (int it = 0; it < KT / kBatch; ++it) {
          const int row = it * kBatch + sub;
          const long long kr = __shfl_sync(0xFFFFFFFFu, ko, row);
          const long long vr = __shfl_sync(0xFFFFFFFFu, vo, row);
          const bool real = (valid >> row) & 1u;
          const uint32_t to = at + row * L::kRow + ((piece ^ (row & 7)) << 4);
          if (has_piece) {
            copy16(to, p.C.k + kr + piece * 16, real);
            copy16(to + KT * L::kRow, p.C.v + vr + piece * 16, real);
          }
        }
        look_up(i + 1);
      }
      copy_commit();
    };
    look_up(u.i0);
#pragma unroll
    for (int s = 0; s < ST - 1; ++s) copy_tile(u.i0 + s);

    // the queries
    const int live = u.live_rows(p);
    for (int i = tid; i < 16 * kPieces; i += kAttnThreads) {
      const int row = i / kPieces, pc = i % kPieces;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (row < live && pc * 8 < p.D) {
        const int r = u.r0 + row, n = r / p.G, g = r - n * p.G;
        x = *reinterpret_cast<const uint4 *>(p.q + u.b * p.q_seq + n * p.q_token +
                                             (u.h * p.G + g) * p.q_head + pc * 16);
      }
      *reinterpret_cast<uint4 *>(q_s + row * L::kRow + ((pc ^ (row & 7)) << 4)) = x;
    }
    __syncthreads();
    uint32_t qf[DP / 16][4];
#pragma unroll
    for (int k = 0; k < DP / 16; ++k) {
      const int row = (lane & 7) + ((lane >> 3) & 1) * 8, pc = k * 2 + (lane >> 4);
      ldsm4(qf[k], q_at + row * L::kRow + ((pc ^ (row & 7)) << 4));
    }
    const int n0 = (u.r0 + min(lane / 4, live - 1)) / p.G;
    const int n1 = (u.r0 + min(lane / 4 + 8, live - 1)) / p.G;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[DP / 8][4];
#pragma unroll
    for (int j = 0; j < DP / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    bool bad = false;

    for (int i = u.i0; i < u.i1; ++i) {
      copy_wait<ST - 2>();
      __syncwarp();
      copy_tile(i + ST - 1);
      const int st = (i - u.i0) % ST;
      const uint32_t valid = valid_s[warp][st];
      if (valid == 0u) continue;
      const int at0 = key_tile(u.k, i) * L::kTile + warp * KT;
      const uint32_t k_at = ring_at + st * L::kStage, v_at = k_at + KT * L::kRow;
      float s[KT / 8][4];
#pragma unroll
      for (int j = 0; j < KT / 8; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
      for (int k = 0; k < DP / 16; ++k) {
#pragma unroll
        for (int j = 0; j < KT / 16; ++j) {
          uint32_t b[4];
          const int row = j * 16 + ((lane >> 4) << 3) + (lane & 7), pc = k * 2 + ((lane >> 3) & 1);
          ldsm4(b, k_at + row * L::kRow + ((pc ^ (row & 7)) << 4));
          mma<E>(s[2 * j], qf[k], b[0], b[1]);
          mma<E>(s[2 * j + 1], qf[k], b[2], b[3]);
        }
      }
      constexpr uint32_t kAll = KT == 32 ? 0xFFFFFFFFu : (1u << KT) - 1u;
      if (valid != kAll || !all_seen(p, u.k, at0, KT)) {
#pragma unroll
        for (int j = 0; j < KT / 8; ++j) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = j * 8 + (lane & 3) * 2 + e;
            const bool there = (valid >> key) & 1u;
            if (!there || !sees(p, u.k, u.b, n0, at0 + key)) s[j][e] = -INFINITY;
            if (!there || !sees(p, u.k, u.b, n1, at0 + key)) s[j][2 + e] = -INFINITY;
          }
        }
        // infinities and NaNs among the values: zero here, see nonfinite_values
        for (int t = lane; t < KT * kPieces; t += 32) {
          uint4 *x = reinterpret_cast<uint4 *>(ring + st * L::kStage + KT * L::kRow + t * 16);
          const uint4 v = make_uint4(finite_or_zero<E>(x->x), finite_or_zero<E>(x->y),
                                     finite_or_zero<E>(x->z), finite_or_zero<E>(x->w));
          if (v.x != x->x || v.y != x->y || v.z != x->z || v.w != x->w) {
            *x = v;
            bad = true;
          }
        }
        __syncwarp();
      }
      float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
      for (int j = 0; j < KT / 8; ++j) {
        x0 = fmaxf(x0, fmaxf(s[j][0], s[j][1]));
        x1 = fmaxf(x1, fmaxf(s[j][2], s[j][3]));
      }
#pragma unroll
      for (int x = 1; x <= 2; x <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, x));
        x1 = fmaxf(x1, __shfl_xor_sync(0xFFFFFFFFu, x1, x));
      }
      // float16 weights are lifted to 2^15, so that those that it rounds to zero are
      // below 2^-40 of the row's largest instead of 2^-25
      constexpr float kLift = E::kNarrow ? 15.f : 0.f;
      x0 = fmaxf(m0, x0 * c - kLift);
      x1 = fmaxf(m1, x1 * c - kLift);
      if (__any_sync(0xFFFFFFFFu, x0 > m0 || x1 > m1)) {
        const float f0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - x0);
        const float f1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - x1);
        m0 = x0;
        m1 = x1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) {
          o[j][0] *= f0;
          o[j][1] *= f0;
          o[j][2] *= f1;
          o[j][3] *= f1;
        }
      }
      // a row that has seen nothing yet keeps weights of zero
      const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
      for (int j = 0; j < KT / 8; ++j) {
        s[j][0] = fast_exp2(fmaf(s[j][0], c, -u0));
        s[j][1] = fast_exp2(fmaf(s[j][1], c, -u0));
        s[j][2] = fast_exp2(fmaf(s[j][2], c, -u1));
        s[j][3] = fast_exp2(fmaf(s[j][3], c, -u1));
        l0 += s[j][0] + s[j][1];
        l1 += s[j][2] + s[j][3];
      }
#pragma unroll
      for (int j = 0; j < KT / 16; ++j) {
        // the matrix product takes the weights in the cache's type: each is off
        // by at most half a step of that type, as the values themselves are
        const uint32_t a[4] = {E::pack(s[2 * j][0], s[2 * j][1]), E::pack(s[2 * j][2], s[2 * j][3]),
                               E::pack(s[2 * j + 1][0], s[2 * j + 1][1]),
                               E::pack(s[2 * j + 1][2], s[2 * j + 1][3])};
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
          uint32_t b[4];
          const int row = j * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), pc = d * 2 + (lane >> 4);
          ldsm4t(b, v_at + row * L::kRow + ((pc ^ (row & 7)) << 4));
          mma<E>(o[2 * d], a, b[0], b[1]);
          mma<E>(o[2 * d + 1], a, b[2], b[3]);
        }
      }
    }

    // the unit's end: the warps' results meet in shared memory
    copy_wait<0>();
    __syncwarp();
#pragma unroll
    for (int x = 1; x <= 2; x <<= 1) {
      l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, x);
      l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, x);
    }
    float *o_w = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int j = 0; j < DP / 8; ++j) {
      const int d = j * 8 + (lane & 3) * 2, row = lane / 4;
      *reinterpret_cast<float2 *>(o_w + row * DP + d) = make_float2(o[j][0], o[j][1]);
      *reinterpret_cast<float2 *>(o_w + (row + 8) * DP + d) = make_float2(o[j][2], o[j][3]);
    }
    if ((lane & 3) == 0) {
      ml_s[warp][0][lane / 4] = m0;
      ml_s[warp][0][lane / 4 + 8] = m1;
      ml_s[warp][1][lane / 4] = l0;
      ml_s[warp][1][lane / 4 + 8] = l1;
    }
    if (bad) bad_s = 1;
    __syncthreads();
    write_unit<TE, 16, DP, KT>(p, u, reinterpret_cast<const float *>(smem + 16 * L::kRow),
                               L::kRing / 4, ml_s, bad_s != 0, line.worker);
    if (!u.next(p, line)) break;
    __syncthreads();
    if (tid == 0) bad_s = 0;
    if (p.D < DP) {
      // the outputs were laid over the pieces that stay zero
      for (int i = lane; i < 16 * DP / 4; i += 32)
        reinterpret_cast<uint4 *>(ring)[i] = make_uint4(0, 0, 0, 0);
      __syncwarp();
    }
  }
}

// ---------------------------------------------------------------------------
// float32, 8 rows per unit
// ---------------------------------------------------------------------------

// A lane takes one of 32 / KT parts of a key of its warp's tile for the scores
// and some of the head's dimensions for the outputs.  Rows of keys are 16 bytes
// longer than their data, so that lanes on different rows meet different banks.
// Bound by shared-memory reads: a key's part is met by eight queries, 9 reads of
// 16 bytes for 32 products.  Tiles of 4 KB a warp leave room for three CTAs an
// SM: 64 sequences of 1 to 4096 tokens, one token each, 32 heads on 8 of 128,
// 244 us (4.4 TB/s); with two CTAs 275, with tiles twice as long and one CTA 350.
template <int DP>
struct Rows8 {
  static constexpr int KT = 1024 / DP;  // 16, 8, 4 keys per warp and tile
  static constexpr int kCtas = DP <= 128 ? 3 : 2;  // of an SM
  static constexpr int ST = 2;
  static constexpr int kTile = kAttnWarps * KT;
  static constexpr int kKeyRow = DP * 4 + 16, kValRow = DP * 4;
  static constexpr int kStage = KT * (kKeyRow + kValRow);
  static constexpr int kRing = ST * kStage;
  static constexpr int kWeights = KT * 8 * 4;
  static constexpr int kSmem = 8 * DP * 4 + kAttnWarps * (kRing + kWeights);
  static_assert(kRing >= 8 * DP * 4, "a warp's outputs fit its ring");
};

template <int DP>
__global__ void __launch_bounds__(kAttnThreads, Rows8<DP>::kCtas) rows8_kernel(const __grid_constant__ AttnParams p) {
  using L = Rows8<DP>;
  constexpr int KT = L::KT, ST = L::ST, R = 8;
  extern __shared__ __align__(128) char smem[];
  __shared__ float ml_s[kAttnWarps][2][R];
  __shared__ uint32_t valid_s[kAttnWarps][ST];
  __shared__ int bad_s;
  __shared__ RunScratch<kAttnThreads, 1> run_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float *q_s = reinterpret_cast<float *>(smem);
  char *rings = smem + R * DP * 4;
  char *ring = rings + warp * L::kRing;
  float *p_s = reinterpret_cast<float *>(rings + kAttnWarps * L::kRing) + warp * KT * R;
  const uint32_t ring_at = smem_u32(ring);
  if (tid == 0) bad_s = 0;
  Line lines[1];
  find_runs(p, run_s, blockIdx.x, 0, lines);
  const Line &line = lines[0];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  UnitWalk u;
  const bool busy = u.start(p, line);
  if (tid == 0) write_join(p, line, busy ? &u : nullptr);
  if (!busy) return;

  constexpr int kPieces = DP / 4;                            // of a row, 16 bytes each
  constexpr int kLanes = kPieces < 32 ? kPieces : 32;        // lanes on one row
  constexpr int kBatch = 32 / kLanes, kOwn = kPieces / kLanes;  // rows at once, pieces a lane
  const int piece = lane % kLanes, sub = lane / kLanes;
  const int pieces = p.D / 4;
  const float c = p.scale_log2;
  const int key = lane % KT, part = lane / KT;

  for (;;) {
    auto copy_tile = [&](int i) {
      if (i < u.i1) {
        const int st = (i - u.i0) % ST;
        const int at = key_tile(u.k, i) * L::kTile + warp * KT + lane;
        int pid = -1, in_page = 0;
        if (lane < KT && at < u.k.end) {
          const int index = at / p.C.page_size;
          in_page = at - index * p.C.page_size;
          pid = page_at(p.S, u.b, index);
        }
        const bool ok = page_ok(p.C, pid);
        const long long ko = ok ? pid * p.C.k_page + in_page * p.C.k_token + u.h * p.C.k_head : 0;
        const long long vo = ok ? pid * p.C.v_page + in_page * p.C.v_token + u.h * p.C.v_head : 0;
        const uint32_t valid = __ballot_sync(0xFFFFFFFFu, ok);
        if (lane == 0) valid_s[warp][st] = valid;
        const uint32_t to = ring_at + st * L::kStage;
#pragma unroll 4
        for (int r0 = 0; r0 < KT; r0 += kBatch) {
          const int row = r0 + sub;
          const long long kr = __shfl_sync(0xFFFFFFFFu, ko, row);
          const long long vr = __shfl_sync(0xFFFFFFFFu, vo, row);
          const bool real = (valid >> row) & 1u;
#pragma unroll
          for (int j = 0; j < kOwn; ++j) {
            const int pc = piece + j * kLanes;
            if (pc < pieces) {
              copy16(to + row * L::kKeyRow + pc * 16, p.C.k + kr + pc * 16, real);
              copy16(to + KT * L::kKeyRow + row * L::kValRow + pc * 16, p.C.v + vr + pc * 16, real);
            }
          }
        }
      }
      copy_commit();
    };
#pragma unroll
    for (int s = 0; s < ST - 1; ++s) copy_tile(u.i0 + s);
    const int live = u.live_rows(p);
    for (int i = tid; i < R * kPieces; i += kAttnThreads) {
      const int row = i / kPieces, pc = i % kPieces;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < live && pc < pieces) {
        const int r = u.r0 + row, n = r / p.G, g = r - n * p.G;
        x = *reinterpret_cast<const float4 *>(p.q + u.b * p.q_seq + n * p.q_token +
                                              (u.h * p.G + g) * p.q_head + pc * 16);
      }
      *reinterpret_cast<float4 *>(q_s + row * DP + pc * 4) = x;
    }
    __syncthreads();
    float m[R], l[R], o[R][4 * kOwn];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int j = 0; j < 4 * kOwn; ++j) o[r][j] = 0.f;
    }
    bool bad = false;

    for (int i = u.i0; i < u.i1; ++i) {
      copy_wait<ST - 2>();
      __syncwarp();
      copy_tile(i + ST - 1);
      const int st = (i - u.i0) % ST;
      const uint32_t valid = valid_s[warp][st];
      if (valid == 0u) continue;
      const int at0 = key_tile(u.k, i) * L::kTile + warp * KT;
      const float *k_s = reinterpret_cast<const float *>(ring + st * L::kStage);
      float *v_s = reinterpret_cast<float *>(ring + st * L::kStage + KT * L::kKeyRow);
      float s[R];
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] = 0.f;
      for (int pc = part; pc < pieces; pc += 32 / KT) {
        const float4 x = *reinterpret_cast<const float4 *>(k_s + key * (L::kKeyRow / 4) + pc * 4);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float4 y = *reinterpret_cast<const float4 *>(q_s + r * DP + pc * 4);
          s[r] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s[r]))));
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int x = KT; x < 32; x <<= 1) s[r] += __shfl_xor_sync(0xFFFFFFFFu, s[r], x);
      constexpr uint32_t kAll = KT == 32 ? 0xFFFFFFFFu : (1u << KT) - 1u;
      if (valid != kAll || !all_seen(p, u.k, at0, KT)) {
        const bool there = (valid >> key) & 1u;
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (!there || !sees(p, u.k, u.b, (u.r0 + min(r, live - 1)) / p.G, at0 + key))
            s[r] = -INFINITY;
        for (int t = lane; t < KT * pieces; t += 32) {
          float4 *x = reinterpret_cast<float4 *>(v_s + t / pieces * DP + t % pieces * 4);
          float4 y = *x;
          float *z = reinterpret_cast<float *>(&y);
          bool found = false;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!isfinite(z[e])) z[e] = 0.f, found = true;
          if (found) *x = y, bad = true;
        }
      }
      bool up = false;
      float f[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float x = s[r];
#pragma unroll
        for (int y = 1; y < KT; y <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, y));
        x = fmaxf(m[r], x * c);
        f[r] = m[r] == -INFINITY ? 0.f : fast_exp2(m[r] - x);
        up |= x > m[r];
        m[r] = x;
        s[r] = fast_exp2(fmaf(s[r], c, x == -INFINITY ? 0.f : -x));
      }
      if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          l[r] *= f[r];
#pragma unroll
          for (int j = 0; j < 4 * kOwn; ++j) o[r][j] *= f[r];
        }
      }
      if (part == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] += s[r];
        *reinterpret_cast<float4 *>(p_s + key * R) = make_float4(s[0], s[1], s[2], s[3]);
        *reinterpret_cast<float4 *>(p_s + key * R + 4) = make_float4(s[4], s[5], s[6], s[7]);
      }
      __syncwarp();
#pragma unroll 4
      for (int k0 = 0; k0 < KT; k0 += kBatch) {
        const int kk = k0 + sub;
        const float4 a = *reinterpret_cast<const float4 *>(p_s + kk * R);
        const float4 b = *reinterpret_cast<const float4 *>(p_s + kk * R + 4);
        const float wt[R] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
          const int pc = piece + j * kLanes;
          if (pc >= pieces) continue;
          const float4 v = *reinterpret_cast<const float4 *>(v_s + kk * DP + pc * 4);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            o[r][4 * j] = fmaf(wt[r], v.x, o[r][4 * j]);
            o[r][4 * j + 1] = fmaf(wt[r], v.y, o[r][4 * j + 1]);
            o[r][4 * j + 2] = fmaf(wt[r], v.z, o[r][4 * j + 2]);
            o[r][4 * j + 3] = fmaf(wt[r], v.w, o[r][4 * j + 3]);
          }
        }
      }
    }

    copy_wait<0>();
    __syncwarp();
    float *o_w = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l[r] = warp_sum(l[r]);
#pragma unroll
      for (int j = 0; j < 4 * kOwn; ++j)
#pragma unroll
        for (int x = kLanes; x < 32; x <<= 1)
          o[r][j] += __shfl_xor_sync(0xFFFFFFFFu, o[r][j], x);
      if (sub == 0) {
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
          store4(o_w + r * DP + (piece + j * kLanes) * 4,
                 make_float4(o[r][4 * j], o[r][4 * j + 1], o[r][4 * j + 2], o[r][4 * j + 3]));
      }
      if (lane == 0) {
        ml_s[warp][0][r] = m[r];
        ml_s[warp][1][r] = l[r];
      }
    }
    if (bad) bad_s = 1;
    __syncthreads();
    write_unit<float, R, DP, KT>(p, u, reinterpret_cast<const float *>(rings), L::kRing / 4, ml_s,
                                 bad_s != 0, line.worker);
    if (!u.next(p, line)) break;
    __syncthreads();
    if (tid == 0) bad_s = 0;
  }
}

// ---------------------------------------------------------------------------
// the join
// ---------------------------------------------------------------------------

// The pieces of a cut unit, of which the worker holds the first; by whole warps.
template <typename TE>
struct Pieces {
  const AttnParams &p;
  const JoinDesc &d;
  int lane, first, lines, count;
  size_t per_slot;
  __device__ __forceinline__ Pieces(const AttnParams &p, const JoinDesc &d, int worker, int lane)
      : p(p), d(d), lane(lane), first(worker - p.row_lines), lines(p.row_lines),
        count((d.pieces_end - first) / lines + 1), per_slot(slot_floats(p.rows, p.D)) {}
  __device__ __forceinline__ const float *slot(int i) const {
    return p.part + (2 * (first + i * lines) + (i == 0 ? 1 : 0)) * per_slot;
  }
  // pieces from, from + step, ... of a row
  __device__ __forceinline__ void gather(int row, int from, int step, float &M, float &l, float4 (&o)[2]) const {
    M = -INFINITY;
    l = 0.f;
    o[0] = o[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = from; i0 < count; i0 += 8 * step) {
      float m[8], lp[8];
      float4 v[8][2];
      float top = M;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + j * step;
        m[j] = -INFINITY;
        lp[j] = 0.f;
        if (i >= count) continue;
        const float *s = slot(i);
        m[j] = s[row];
        lp[j] = s[p.rows + row];
        const float *from_o = s + slot_stats(p.rows) + static_cast<size_t>(row) * p.D;
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if ((lane + 32 * x) * 4 < p.D)
            v[j][x] = *reinterpret_cast<const float4 *>(from_o + (lane + 32 * x) * 4);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, m[j]);
      if (M > -INFINITY && top > M) {
        const float f = fast_exp2(M - top);
        l *= f;
#pragma unroll
        for (int x = 0; x < 2; ++x) o[x].x *= f, o[x].y *= f, o[x].z *= f, o[x].w *= f;
      }
      M = top;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (lp[j] == 0.f) continue;
        const float f = fast_exp2(m[j] - M);
        l += f * lp[j];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if ((lane + 32 * x) * 4 >= p.D) continue;
          o[x].x += f * v[j][x].x;
          o[x].y += f * v[j][x].y;
          o[x].z += f * v[j][x].z;
          o[x].w += f * v[j][x].w;
        }
      }
    }
  }
  __device__ __forceinline__ void finish(int row, float M, float l, const float4 (&o)[2]) const {
    const long long at = out_row(p, d.b, d.h, d.r0 + row);
    const float r = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int e = (lane + 32 * x) * 4;
      if (e < p.D)
        store4(static_cast<TE *>(p.out) + at * p.D + e,
               make_float4(o[x].x * r, o[x].y * r, o[x].z * r, o[x].w * r));
    }
    if (lane == 0 && p.lse) p.lse[at] = row_lse(M, l);
  }
};

// The rows of a cut unit, dealt over gridDim.y CTAs.  Units of two pieces, the
// most there are in a full batch: a warp takes four rows at once, since a row
// alone is one round trip to L2 whatever its size.  Units of few pieces: a warp
// per row.  Units of many: the CTA's warps share the pieces of one row after the
// other, and their sums are added in order.  A warp has eight pieces in flight.
template <class TE>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ float m_s[kWarps], l_s[kWarps];
  __shared__ float4 o_s[kWarps][64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const JoinDesc d = p.join[blockIdx.x];
  if (d.pieces_end < 0) return;
  const int rows = d.rows, Y = gridDim.y;
  const Pieces<TE> u(p, d, blockIdx.x, lane);
  const int count = u.count;
  if (count == 2 && p.D <= 128) {
    const float *s[2] = {u.slot(0), u.slot(1)};
    const int at = lane * 4;
    for (int r = (blockIdx.y * kWarps + warp) * 4; r < rows; r += 4 * Y * kWarps) {
      float m[4][2], l[4][2];
      float4 v[4][2];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = min(r + j, rows - 1);
          m[j][x] = s[x][row];
          l[j][x] = s[x][p.rows + row];
          if (at < p.D)
            v[j][x] = *reinterpret_cast<const float4 *>(s[x] + slot_stats(p.rows) +
                                                        static_cast<size_t>(row) * p.D + at);
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = r + j;
        if (row >= rows) break;
        const float M = fmaxf(m[j][0], m[j][1]);
        float f[2], sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (l[j][x] == 0.f) continue;
          f[x] = fast_exp2(m[j][x] - M);
          sum += f[x] * l[j][x];
          o.x += f[x] * v[j][x].x;
          o.y += f[x] * v[j][x].y;
          o.z += f[x] * v[j][x].z;
          o.w += f[x] * v[j][x].w;
        }
        const long long to = out_row(p, d.b, d.h, d.r0 + row);
        const float n = sum == 0.f ? 0.f : 1.f / sum;
        if (at < p.D)
          store4(static_cast<TE *>(p.out) + to * p.D + at,
                 make_float4(o.x * n, o.y * n, o.z * n, o.w * n));
        if (lane == 0 && p.lse) p.lse[to] = row_lse(M, sum);
      }
    }
    return;
  }
  float M, l;
  float4 o[2];
  if (count <= 16) {
    for (int row = blockIdx.y * kWarps + warp; row < rows; row += Y * kWarps) {
      u.gather(row, 0, 1, M, l, o);
      u.finish(row, M, l, o);
    }
    return;
  }
  for (int row = blockIdx.y; row < rows; row += Y) {
    u.gather(row, warp, kWarps, M, l, o);
    if (lane == 0) {
      m_s[warp] = M;
      l_s[warp] = l;
    }
    o_s[warp][lane] = o[0];
    o_s[warp][lane + 32] = o[1];
    __syncthreads();
    if (warp == 0) {
      M = fmaxf(fmaxf(m_s[0], m_s[1]), fmaxf(m_s[2], m_s[3]));
      l = 0.f;
      o[0] = o[1] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (l_s[w] == 0.f) continue;
        const float f = fast_exp2(m_s[w] - M);
        l += f * l_s[w];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float4 v = o_s[w][lane + 32 * x];
          o[x].x += f * v.x;
          o[x].y += f * v.y;
          o[x].z += f * v.z;
          o[x].w += f * v.w;
        }
      }
      u.finish(row, M, l, o);
    }
    __syncthreads();
  }
}

// For few units cut into many pieces by many workers, most of which have no unit to join:
// a CTA looks at 32 of them.  Their units of few pieces are dealt over its warps row by row;
// the pieces of larger ones are shared by all warps, a row after the other.  (1824 workers,
// both kernels of a call together, a CTA a worker and 32: 8 units of 32 tiles 16.4 us and
// 13.2, 8 of about 3000 tiles, 7 rows 58.7 and 45.2, but 2048 units 158 and 166.)
constexpr int kManyThreads = 512, kManyWorkers = 32, kFewPieces = 16;
template <typename TE>
__global__ void __launch_bounds__(kManyThreads) join_many_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kWarps = kManyThreads / 32;
  __shared__ float m_s[kWarps], l_s[kWarps];
  __shared__ float4 o_s[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, Y = gridDim.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int worker0 = blockIdx.x * kManyWorkers;
  // a worker's unit a lane
  JoinDesc mine = {0, 0, 0, 0, -1};
  if (worker0 + lane < p.workers) mine = p.join[worker0 + lane];
  const int count = mine.pieces_end < 0 ? 0 : Pieces<TE>(p, mine, worker0 + lane, lane).count;
  auto unit_of = [&](int of) {
    return JoinDesc{__shfl_sync(0xFFFFFFFFu, mine.b, of), __shfl_sync(0xFFFFFFFFu, mine.h, of),
                    __shfl_sync(0xFFFFFFFFu, mine.r0, of), __shfl_sync(0xFFFFFFFFu, mine.rows, of),
                    __shfl_sync(0xFFFFFFFFu, mine.pieces_end, of)};
  };
  float M, l;
  float4 o[2];
  int turn = 0;
  for (uint32_t left = __ballot_sync(0xFFFFFFFFu, count > 0 && count <= kFewPieces); left; left &= left - 1) {
    const int worker = worker0 + __ffs(left) - 1;
    const JoinDesc d = unit_of(worker - worker0);
    const Pieces<TE> u(p, d, worker, lane);
    for (int row = blockIdx.y; row < d.rows; row += Y) {
      if (turn++ % kWarps != warp) continue;
      u.gather(row, 0, 1, M, l, o);
      u.finish(row, M, l, o);
    }
  }
  for (uint32_t left = __ballot_sync(0xFFFFFFFFu, count > kFewPieces); left; left &= left - 1) {
    const int worker = worker0 + __ffs(left) - 1;
    const JoinDesc d = unit_of(worker - worker0);
    const Pieces<TE> u(p, d, worker, lane);
    for (int row = blockIdx.y; row < d.rows; row += Y) {
      u.gather(row, warp, kWarps, M, l, o);
      if (lane == 0) {
        m_s[warp] = M;
        l_s[warp] = l;
      }
      o_s[warp][lane] = o[0];  // head dimensions up to 128
      __syncthreads();
      if (warp == 0) {
        M = -INFINITY;
        l = 0.f;
        o[0] = o[1] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, m_s[w]);
        for (int w = 0; w < kWarps; ++w) {
          if (l_s[w] == 0.f) continue;
          const float f = fast_exp2(m_s[w] - M);
          l += f * l_s[w];
          const float4 v = o_s[w][lane];
          o[0].x += f * v.x;
          o[0].y += f * v.y;
          o[0].z += f * v.z;
          o[0].w += f * v.w;
        }
        u.finish(row, M, l, o);
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------

// AttnPlan::few.
// Units of at most so many tiles are not cut: one launch for two (4.4 us of the
// caller's time) and no join (3 to 5 us), against tiles that follow each other on
// one worker.  From both forms at B = 1, 16 and 64 over 32 to 8192 keys, contexts of
// one length and of 1/16 of it upwards, us cut and whole: one token of 32 heads of
// 128 on 8, 512 keys 12.0, 12.4 (B = 1) and 36.2, 30.8 (B = 64), 1024 keys 12.6, 16.7
// and 56, 51, ragged 39, 43; trees of 60 nodes, 1024 keys 26, 24 (B = 1) and 40, 27
// (B = 16), 2048 keys 36, 37 and 61, 44, 4096 keys 37, 62.  Borders that move to the
// ends of longer units did not pay.

constexpr int log2_of(int x) { return x <= 1 ? 0 : 1 + log2_of(x / 2); }

AttnPlan narrow_plan(int D, int dtype) {
  if (dtype == SPEC_F32) {
    if (D <= 64) return {Rows8<64>::kCtas * kSms, 8, log2_of(Rows8<64>::kTile), 1, 2};
    if (D <= 128) return {Rows8<128>::kCtas * kSms, 8, log2_of(Rows8<128>::kTile), 1, 2};
    return {Rows8<256>::kCtas * kSms, 8, log2_of(Rows8<256>::kTile), 1, 2};
  }
  if (D <= 64) return {2 * kSms, 16, log2_of(Rows16<64, 32, 3>::kTile), 1, 4};
  if (D <= 128) return {2 * kSms, 16, log2_of(Rows16<128, 16, 3>::kTile), 1, 4};
  return {kSms, 16, log2_of(Rows16<256, 16, 3>::kTile), 1, 2};
}

// Lines of 19 workers each at least; 152 are a multiple of 2, 4 and 8.
constexpr int kMaxRowLines = 8;

bool wide_sizes(int G, int D, int dtype) {
  return dtype != SPEC_F32 && (D == 64 || D == 128) && G <= 128;
}
// What a unit costs beside its tiles (queries, the first products and the last,
// masked tiles, outputs), in tiles, from runs of one launch fitted by their tiles
// and units: pairs of row tiles 8 (12 to 16 us; 256-node trees at B=16 and 60-node
// ones at B=32 take 517 and 114 us with 5, 517 and 111 with 7, 523 and 111 with 8, 525
// and 111 with 9, 529 and 109 with 10), single ones 1 at head_dim 128, where HBM hides
// it, and 2 at 64.
AttnPlan wide_plan(int N, int G, int D) {
  if (N * G > wide_tile_rows(G)) return {kSms, 2 * wide_tile_rows(G), 7, 8, 16};
  return {2 * kSms, wide_tile_rows(G), 7, D == 64 ? 2 : 1, N * G <= 32 ? 4 : 6};
}

template <auto kKernel>
cudaError_t start(size_t smem, const AttnParams &p, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  return launch_large(kKernel, done, static_cast<int>(smem), p.workers, kAttnThreads,
                      static_cast<int>(smem), stream, p);
}

template <class E>
cudaError_t start16(const AttnParams &p, cudaStream_t stream) {
  if (p.D <= 64) return start<rows16_kernel<E, 64, 32, 3>>(Rows16<64, 32, 3>::kSmem, p, stream);
  if (p.D <= 128) return start<rows16_kernel<E, 128, 16, 3>>(Rows16<128, 16, 3>::kSmem, p, stream);
  return start<rows16_kernel<E, 256, 16, 3>>(Rows16<256, 16, 3>::kSmem, p, stream);
}

// Whether units are not cut: the width of the page table, or the window, bounds
// their tiles by `few`.  The lengths themselves are known on the device alone.
bool whole_units(const AttnParams &p, int few) {
  const int log2 = p.tile_log2, round = (1 << log2) - 1;
  long long tiles = (static_cast<long long>(p.S.max_pages) * p.C.page_size + round) >> log2;
  if (p.window) {
    const long long sinks = std::min((static_cast<long long>(p.sinks) + round) >> log2, tiles);
    tiles = std::min(tiles, sinks + ((static_cast<long long>(p.window) + p.S.N) >> log2) + 2);
  }
  return tiles <= few;
}

size_t align32(size_t x) { return (x + 31) / 32 * 32; }

}  // namespace

size_t plan_bytes(const AttnPlan &plan, int D) {
  return align32(plan.workers * sizeof(JoinDesc)) +
         2 * plan.workers * slot_floats(plan.rows, D) * sizeof(float);
}

size_t attention_workspace_bytes(int N, int G, int D, int dtype) {
  const size_t narrow = plan_bytes(narrow_plan(D, dtype), D);
  const size_t wide = wide_sizes(G, D, dtype) ? plan_bytes(wide_plan(N, G, D), D) : 0;
  return narrow > wide ? narrow : wide;
}

void take_plan(AttnParams &p, const AttnPlan &plan, void *workspace) {
  p.workers = plan.workers;
  p.rows = plan.rows;
  p.tile_log2 = plan.tile_log2;
  p.unit_cost = plan.unit_cost;
  p.whole = whole_units(p, plan.few);
  p.row_lines = 1;
  p.join = static_cast<JoinDesc *>(workspace);
  p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                     align32(p.workers * sizeof(JoinDesc)));
}

template <typename TE>
cudaError_t start_join(const AttnParams &p, cudaStream_t stream) {
  const int rows = std::min(8, std::min(p.rows, p.S.N * p.G));
  const int tiles = (p.S.N * p.G + p.rows - 1) / p.rows;
  if constexpr (sizeof(TE) == 2)
    if (p.workers > 8 * kSms && p.workers > 4ll * p.S.B * p.C.heads * tiles && p.D <= 128) return launch_behind(
        join_many_kernel<TE>, dim3((p.workers + kManyWorkers - 1) / kManyWorkers, rows), kManyThreads, 0, stream, p);
  // many workers have few rows each: a warp a row (1824 workers, one token at B = 256 155 us, with
  // four blocks for the four rows 158; two tokens, eight rows, at B = 64 63.6 us and 68.8)
  return launch_behind(join_kernel<TE>, dim3(p.workers, p.workers > 8 * kSms ? (rows + 3) / 4 : rows), kJoinThreads,
                       0, stream, p);
}
cudaError_t launch_join(const AttnParams &p, int dtype, cudaStream_t stream) {
  if (dtype == SPEC_F32) return start_join<float>(p, stream);
  return dtype == SPEC_BF16 ? start_join<__nv_bfloat16>(p, stream) : start_join<__half>(p, stream);
}

cudaError_t launch_attention(AttnParams &p, int dtype, void *workspace, cudaStream_t stream) {
  const int P = p.C.page_size;
  WideMaps maps;
  bool wide = wide_sizes(p.G, p.D, dtype) && P % 8 == 0;
  if (wide) {
    take_plan(p, wide_plan(p.S.N, p.G, p.D), workspace);
    // row tiles of a tree see the same keys; those of a chain end at their own
    const int tiles = (p.S.N * p.G + p.rows - 1) / p.rows;
    if (p.mask && tiles <= kMaxRowLines) p.row_lines = tiles;
    wide = wide_maps(p, dtype, &maps);
  }
  if (!wide) take_plan(p, narrow_plan(p.D, dtype), workspace);
  cudaError_t e;
  if (dtype == SPEC_F32) {
    if (p.D <= 64) {
      e = start<rows8_kernel<64>>(Rows8<64>::kSmem, p, stream);
    } else if (p.D <= 128) {
      e = start<rows8_kernel<128>>(Rows8<128>::kSmem, p, stream);
    } else {
      e = start<rows8_kernel<256>>(Rows8<256>::kSmem, p, stream);
    }
  } else if (wide) {
    e = launch_attention_wide(p, maps, dtype, stream);
  } else {
    e = dtype == SPEC_BF16 ? start16<Bf16>(p, stream) : start16<F16>(p, stream);
  }
  if (e != cudaSuccess || p.whole) return e;
  return launch_join(p, dtype, stream);
}

}  // namespace sv
