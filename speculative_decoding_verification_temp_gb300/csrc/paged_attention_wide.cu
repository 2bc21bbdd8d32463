// Attention of many rows over a paged cache: 16-bit types, head_dim 64 or 128,
// units of 128 or 256 rows (new tokens times the query heads of a group) on the
// fifth-generation tensor cores.
//
// Two streams of work share a CTA: with 256 rows each takes half of the rows
// and all key tiles, with 128 rows each takes all rows and every second key
// tile, and their results are added at the end.  For a tile of 128 keys a
// stream computes S = Q K^T into tensor memory (128 lanes of rows x 128
// columns), one thread per row turns S into weights in place (the running
// maximum, the sum, 2^(s c - m) packed into the first half of S's columns), and
// O += P V takes them from there as the A operand.  While one stream is in its
// softmax the other's products run.
//
// Warps 0-3 and 4-7: the softmax of stream 0 and 1.  Warps 8-11: queries, keys
// and values into shared memory, 16 bytes a copy, so that a tile's rows may lie
// on any pages; a ring of entries of 128 rows, keys and values in turn.  One
// thread of warp 12 issues every product.  Copies and products meet at
// mbarriers; every wait is bounded.
//
// Shared rows are 128-byte pieces in the 128-byte swizzle, panels of 64
// elements one behind another: rows of K are K-major for S = Q K^T, rows of V
// are N-major for O += P V, without a transpose.
#include "paged_attention.cuh"

namespace sv {

namespace {

constexpr int kSoft = 256;              // softmax threads
constexpr int kLoad = 128;              // copying threads
constexpr int kWideThreads = kSoft + kLoad + 32;
constexpr int kTileKeys = 128;
constexpr int kValidRing = 16;
constexpr long long kWaitCycles = 4000000000ll;  // about two seconds
// The running maximum is raised only when a row's scores pass it by this much
// (in powers of two): until then weights stay below 2^8 and no output is
// rescaled.  Weights above one have the same relative rounding.
constexpr float kSlack = 8.f;

template <int D, int NQ>
struct WideShape {
  static constexpr int kRow = 128;                    // bytes of a row in a panel
  static constexpr int kPanel = kTileKeys * kRow;     // 128 rows of 64 elements
  static constexpr int kPanels = D / 64;
  static constexpr int kEntry = kPanels * kPanel;
  static constexpr int kQ = NQ * kEntry;
  // what 227 KB hold beside the queries
  static constexpr int kRing = D == 128 ? (NQ == 2 ? 5 : 6) : (NQ == 2 ? 10 : 12);
  static constexpr int kLag = kRing - 2;              // entries in flight before a wait
};

template <int NQ>
struct WideCtl {
  unsigned long long full[12], empty[12], s_full[2], p_full[2], o_done[2], q_full, q_empty, meet,
      drain;
  long long warp_s[kWideThreads / 32], found_s[2];
  alignas(16) uint32_t valid[kValidRing][4];
  uint32_t fix[4][12];
  uint32_t tmem;
  int dead, bad;
  float ml[NQ == 1 ? 2 : 1][2][NQ == 1 ? 128 : 1];
};

template <int D, int NQ>
constexpr int wide_smem() {
  return WideShape<D, NQ>::kQ + WideShape<D, NQ>::kRing * WideShape<D, NQ>::kEntry +
         static_cast<int>(sizeof(WideCtl<NQ>));
}
static_assert(wide_smem<128, 2>() <= 227 * 1024 && wide_smem<128, 1>() <= 227 * 1024 &&
                  wide_smem<64, 2>() <= 227 * 1024 && wide_smem<64, 1>() <= 227 * 1024,
              "shared memory of a CTA");

__device__ __forceinline__ void bar_init(const void *bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(const void *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// Waits for the phase of this parity; gives up after kWaitCycles, or when
// another thread of the CTA has given up.
__device__ __forceinline__ bool bar_wait(const void *bar, uint32_t parity, int *dead) {
  const uint32_t at = smem_u32(bar);
  if (bar_test(at, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    for (int i = 0; i < 16; ++i)
      if (bar_test(at, parity)) return true;
    if (*reinterpret_cast<volatile int *>(dead)) return false;
    if (clock64() - t0 > kWaitCycles) {
      *reinterpret_cast<volatile int *>(dead) = 1;
      return false;
    }
  }
}

// The same by a whole warp, which goes on together.
__device__ __forceinline__ bool warp_wait(const void *bar, uint32_t parity, int *dead) {
  return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, dead));
}

__device__ __forceinline__ void mma_commit(const void *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}
// D (+)= A B, A and B in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add ? 1 : 0)
      : "memory");
}
// A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tm_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tm_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 32 columns of this thread's lane.
__device__ __forceinline__ void tm_load32(uint32_t (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tm_store32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tm_store16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Shared-memory matrix descriptor: 128-byte swizzle; `lead` and `stride` are
// byte distances (between 64-element panels of an N-major operand; between
// groups of eight rows).
__device__ __forceinline__ uint64_t smem_desc(uint32_t at, uint32_t lead, uint32_t stride) {
  return static_cast<uint64_t>((at >> 4) & 0x3FFFu) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(stride >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: 128 rows, n columns, float32 sums; b_n_major: B rows
// run along n.
template <class E>
__device__ __forceinline__ constexpr uint32_t mma_idesc(int n, bool b_n_major);
template <>
__device__ __forceinline__ constexpr uint32_t mma_idesc<Bf16>(int n, bool b_n_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_n_major ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
template <>
__device__ __forceinline__ constexpr uint32_t mma_idesc<F16>(int n, bool b_n_major) {
  return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (8u << 24);
}

__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// Which of the 32 keys from `at` on token n sees (sees() for all of them), of
// those in `valid`.
__device__ __forceinline__ uint32_t seen_word(const AttnParams &p, const KeyRange &k, int b, int n,
                                              int at, uint32_t valid) {
  const uint32_t in_ctx = low_bits(k.ctx - at);
  uint32_t w = valid & in_ctx, block = valid & ~in_ctx;
  const int place = p.window ? k.ctx + clamp_pos(p, b, n) : 0;
  if (p.window) w &= low_bits(p.sinks - at) | ~low_bits(place - p.window + 1 - at);
  if (block) {
    const int m0 = at - k.ctx;  // above -32
    block &= low_bits(k.n_new - m0);
    if (p.mask) {
      const unsigned long long *row = reinterpret_cast<const unsigned long long *>(p.mask) +
                                      static_cast<long long>(b) * p.mask_seq +
                                      static_cast<long long>(n) * p.words;
      unsigned long long bits = 0ull;
      if (m0 < 0) {
        bits = __ldg(row) << -m0;
      } else if ((m0 >> 6) < p.words) {
        bits = __ldg(row + (m0 >> 6)) >> (m0 & 63);
        if ((m0 & 63) > 32 && (m0 >> 6) + 1 < p.words)
          bits |= __ldg(row + (m0 >> 6) + 1) << (64 - (m0 & 63));
      }
      block &= static_cast<uint32_t>(bits);
    } else {
      block &= low_bits(n + 1 - m0);
    }
    if (p.window) {
      for (uint32_t left = block; left; left &= left - 1) {
        const int j = __ffs(left) - 1;
        const int q = k.ctx + clamp_pos(p, b, m0 + j);
        if (q >= p.sinks && place - q >= p.window) block &= ~(1u << j);
      }
    }
  }
  return w | block;
}

}  // namespace

template <class E, int D, int NQ>
__global__ void __launch_bounds__(kWideThreads, 1) wide_kernel(const __grid_constant__ AttnParams p) {
  using W = WideShape<D, NQ>;
  using TE = typename E::T;
  // all shared memory is this array, so its alignment is the swizzle's
  extern __shared__ __align__(1024) char wide_s[];
  char *smem = wide_s;
  char *q_s = smem, *ring = smem + W::kQ;
  WideCtl<NQ> &ctl = *reinterpret_cast<WideCtl<NQ> *>(ring + W::kRing * W::kEntry);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);

  if (tid == 0) {
    for (int i = 0; i < W::kRing; ++i) {
      bar_init(&ctl.full[i], 4);
      bar_init(&ctl.empty[i], 1);
    }
    for (int g = 0; g < 2; ++g) {
      bar_init(&ctl.s_full[g], 1);
      bar_init(&ctl.p_full[g], 128);
      bar_init(&ctl.o_done[g], 1);
    }
    bar_init(&ctl.q_full, 4);
    bar_init(&ctl.q_empty, 1);
    bar_init(&ctl.meet, kSoft);
    bar_init(&ctl.drain, 1);
    ctl.dead = 0;
    ctl.bad = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const Line line = find_run<kWideThreads>(p, ctl.warp_s, ctl.found_s);  // also a barrier
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (line.w0 == line.w1) {
    if (tid == 0) write_join(p, line, nullptr);
    return;
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&ctl.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = ctl.tmem;
  UnitWalk u;
  u.start(p, line);
  if (tid == 0) write_join(p, line, &u);

  if (warp < 8) {
    // -------------------------------------------------------------- softmax
    const int g = warp >> 2;
    const int lane_row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + g * 128, o_at = tmem + lanes + 256;
    const float c = p.scale_log2;
    uint32_t n_s = 0, n_o[2] = {0, 0}, n_meet = 0;
    int tiles_before = 0;  // of this CTA, for the ring of validity words
    bool ok = true;
    for (long long w = line.w0; ok;) {
      const int n_tiles = u.i1 - u.i0, live = u.live_rows(p);
      const int row = NQ == 2 ? g * 128 + lane_row : lane_row;
      const int n = (u.r0 + min(row, live - 1)) / p.G;
      const bool active = NQ == 1 || g * 128 < live;
      float m = -INFINITY, l = 0.f;
      for (int i = NQ == 2 ? 0 : g; active && i < n_tiles; i += NQ == 2 ? 1 : 2) {
        if (!(ok = warp_wait(&ctl.s_full[g], n_s++ & 1u, &ctl.dead))) break;
        tc_after();
        const int at0 = key_tile(u.k, u.i0 + i) * kTileKeys;
        const uint4 valid =
            *reinterpret_cast<const uint4 *>(ctl.valid[(tiles_before + i) % kValidRing]);
        const bool masked = (valid.x & valid.y & valid.z & valid.w) != 0xFFFFFFFFu ||
                            !all_seen(p, u.k, u.r0, at0, kTileKeys);
        uint32_t vis[4] = {valid.x, valid.y, valid.z, valid.w};
        if (masked) {
#pragma unroll
          for (int j = 0; j < 4; ++j) vis[j] = seen_word(p, u.k, u.b, n, at0 + j * 32, vis[j]);
        }
        float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t s[32];
          tm_load32(s, s_at + j * 32);
          tm_wait_ld();
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((vis[j] >> e) & 1u)) s[e] = __float_as_uint(-INFINITY);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e & 3] = fmaxf(x[e & 3], __uint_as_float(s[e]));
        }
        const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * c;
        const bool raise = top > m + kSlack || (m == -INFINITY && top > m);
        if (__any_sync(0xFFFFFFFFu, raise)) {
          const float to = raise ? top : m;
          const float f = m == -INFINITY ? 0.f : fast_exp2(m - to);
          l *= f;
          m = to;
          if (i >= (NQ == 2 ? 1 : 2)) {
            // the products before S's are complete: O is whole
#pragma unroll
            for (int d = 0; d < D / 32; ++d) {
              uint32_t o[32];
              tm_load32(o, o_at + g * 128 + d * 32);
              tm_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tm_store32(o_at + g * 128 + d * 32, o);
            }
          }
        }
        const float sub = m == -INFINITY ? 0.f : -m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t s[32], packed[16];
          tm_load32(s, s_at + j * 32);
          tm_wait_ld();
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((vis[j] >> e) & 1u)) s[e] = __float_as_uint(-INFINITY);
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float a = fast_exp2(fmaf(__uint_as_float(s[e]), c, sub));
            const float b = fast_exp2(fmaf(__uint_as_float(s[e + 1]), c, sub));
            sum[e & 2] += a;
            sum[(e & 2) + 1] += b;
            // the product takes the weights in the cache's type: each is off by
            // at most half a step of that type, as the values themselves are
            packed[e / 2] = E::pack(a, b);
          }
          tm_store16(s_at + j * 16, packed);  // over columns that have been read
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tm_wait_st();
        tc_before();
        bar_arrive(&ctl.p_full[g]);
      }
      if (!ok) break;
      tiles_before += n_tiles;

      // the unit's end
      const bool has1 = NQ == 2 ? live > 128 : n_tiles > 1;
      const bool whole = u.whole();
      float *slot = p.part + piece_slot(u) * slot_floats(p.rows, D);
      const bool mine = row < live;
      const long long out_at = mine ? out_row(p, u.b, u.h, u.r0 + row) : 0;
      const int d_from = NQ == 2 ? 0 : g * (D / 2), d_to = NQ == 2 ? D : d_from + D / 2;
      float w0 = 1.f, w1 = 0.f;  // weights of the streams' outputs
      if constexpr (NQ == 2) {
        if (active) {
          ok = warp_wait(&ctl.o_done[g], n_o[g]++ & 1u, &ctl.dead);
          if (!ok) break;
        }
      } else {
        ctl.ml[g][0][lane_row] = m;
        ctl.ml[g][1][lane_row] = l;
        bar_arrive(&ctl.meet);
        if (!(ok = warp_wait(&ctl.meet, n_meet++ & 1u, &ctl.dead))) break;
        if (!(ok = warp_wait(&ctl.o_done[0], n_o[0]++ & 1u, &ctl.dead))) break;
        if (has1 && !(ok = warp_wait(&ctl.o_done[1], n_o[1]++ & 1u, &ctl.dead))) break;
        const float m0 = ctl.ml[0][0][lane_row], m1 = ctl.ml[1][0][lane_row];
        m = fmaxf(m0, m1);
        w0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - m);
        w1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - m);
        l = (w0 > 0.f ? w0 * ctl.ml[0][1][lane_row] : 0.f) +
            (w1 > 0.f ? w1 * ctl.ml[1][1][lane_row] : 0.f);
        // NaN weights (an infinite maximum) go through
        if (w0 != w0 || w1 != w1) l = w0 + w1;
      }
      if (active) {
        tc_after();
        const float norm = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        const bool bad = *reinterpret_cast<volatile int *>(&ctl.bad) != 0;
#pragma unroll 1
        for (int d = d_from; d < d_to; d += 32) {
          __syncwarp();
          uint32_t o[32];
          tm_load32(o, o_at + (NQ == 2 ? g * 128 : 0) + d);
          tm_wait_ld();
          if constexpr (NQ == 1) {
            uint32_t o1[32];
            tm_load32(o1, o_at + 128 + d);
            tm_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float a = w0 == 0.f ? 0.f : w0 * __uint_as_float(o[e]);
              const float b = w1 == 0.f ? 0.f : w1 * __uint_as_float(o1[e]);
              o[e] = __float_as_uint(a + b);
            }
          }
          if (!mine) continue;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float4 v = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                   __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
            if (l == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (bad) v = nonfinite_values<TE, 32>(p, u, n, d + e, v);
            if (whole) {
              v = make_float4(v.x * norm, v.y * norm, v.z * norm, v.w * norm);
              store4(static_cast<TE *>(p.out) + out_at * D + d + e, v);
            } else {
              store4(slot + 2 * p.rows + static_cast<size_t>(row) * D + d + e, v);
            }
          }
        }
        if (mine && d_from == 0) {
          if (!whole) {
            slot[row] = m;
            slot[p.rows + row] = l;
          } else if (p.lse) {
            p.lse[out_at] = row_lse(m, l);
          }
        }
        __syncwarp();
        tc_before();
      }
      if constexpr (NQ == 1) {
        // both halves have been read before either stream's next output begins
        bar_arrive(&ctl.meet);
        if (!(ok = warp_wait(&ctl.meet, n_meet++ & 1u, &ctl.dead))) break;
      }
      w += n_tiles;
      if (w >= line.w1) break;
      u.next(p, line);
    }
  } else if (warp < 12) {
    // --------------------------------------------------------------- copies
    const int wl = warp - 8;
    constexpr int kPieces = D / 8, kBatch = 32 / kPieces;  // 16-byte pieces, rows at once
    const int piece = lane % kPieces, sub = lane / kPieces;
    const uint32_t ring_at = smem_u32(ring), q_at = smem_u32(q_s);
    // piece's place in row r of an entry: panel, row, swizzled 16 bytes
    auto place = [&](int r, int pc) {
      return static_cast<uint32_t>((pc >> 3) * W::kPanel + r * W::kRow + (((pc & 7) ^ (r & 7)) << 4));
    };
    uint32_t put = 0, told = 0;  // entries copied to, entries announced
    int tiles_before = 0;
    bool ok = true;

    // Announces the oldest entry that is not yet: its copies have landed.
    auto tell = [&]() {
      const int slot = told % W::kRing;
      if (ctl.fix[wl][slot]) {
        bool found = false;
        for (int t = lane; t < 32 * kPieces; t += 32) {
          uint4 *x = reinterpret_cast<uint4 *>(
              ring + slot * W::kEntry + place(wl * 32 + t / kPieces, t % kPieces));
          const uint4 v = make_uint4(finite_or_zero<E>(x->x), finite_or_zero<E>(x->y),
                                     finite_or_zero<E>(x->z), finite_or_zero<E>(x->w));
          if (v.x != x->x || v.y != x->y || v.z != x->z || v.w != x->w) {
            *x = v;
            found = true;
          }
        }
        if (found) *reinterpret_cast<volatile int *>(&ctl.bad) = 1;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive(&ctl.full[slot]);
      ++told;
    };
    auto flush = [&]() {
      copy_wait<0>();
      __syncwarp();  // fixes read pieces that other lanes have copied
      while (told < put) tell();
    };
    // Copies this warp's 32 rows of the keys or values of tile i of the unit.
    auto copy_entry = [&](bool values, int i) {
      const int slot = put % W::kRing;
      if (!(ok = warp_wait(&ctl.empty[slot], ((put / W::kRing) & 1u) ^ 1u, &ctl.dead))) return;
      const int at0 = key_tile(u.k, u.i0 + i) * kTileKeys + wl * 32, at = at0 + lane;
      long long off = 0;
      bool there = false;
      if (at < u.k.end) {
        const int index = at / p.C.page_size, page = page_at(p.S, u.b, index);
        there = page_ok(p.C, page);
        if (there)
          off = values ? page * p.C.v_page + (at - index * p.C.page_size) * p.C.v_token + u.h * p.C.v_head
                       : page * p.C.k_page + (at - index * p.C.page_size) * p.C.k_token + u.h * p.C.k_head;
      }
      const uint32_t valid = __ballot_sync(0xFFFFFFFFu, there);
      if (lane == 0) {
        if (!values) ctl.valid[(tiles_before + i) % kValidRing][wl] = valid;
        ctl.fix[wl][slot] =
            values && valid != 0u && (valid != 0xFFFFFFFFu || !all_seen(p, u.k, u.r0, at0, 32));
      }
      __syncwarp();
      const char *base = values ? p.C.v : p.C.k;
      const uint32_t to = ring_at + slot * W::kEntry;
#pragma unroll 8
      for (int it = 0; it < 32 / kBatch; ++it) {
        const int r = it * kBatch + sub;
        const long long o = __shfl_sync(0xFFFFFFFFu, off, r);
        copy16(to + place(wl * 32 + r, piece), base + o + piece * 16, (valid >> r) & 1u);
      }
      copy_commit();
      ++put;
      if (put - told > W::kLag) {
        copy_wait<W::kLag>();
        __syncwarp();
        tell();
      }
    };

    uint32_t n_q = 0;
    for (long long w = line.w0; ok;) {
      const int n_tiles = u.i1 - u.i0, live = u.live_rows(p);
      // entries in the order in which the products need them
      if constexpr (NQ == 2) {
        copy_entry(false, 0);
        if (ok) copy_entry(true, 0);
      } else {
        copy_entry(false, 0);
        if (ok && n_tiles > 1) copy_entry(false, 1);
      }
      if (!ok) break;
      flush();
      // the queries, once the products of the unit before have read theirs
      if (!(ok = warp_wait(&ctl.q_empty, (n_q++ & 1u) ^ 1u, &ctl.dead))) break;
#pragma unroll 4
      for (int it = 0; it < NQ * 32 / kBatch; ++it) {
        const int r = (it * 4 + wl) * kBatch + sub;
        const bool there = r < live;
        const int f = u.r0 + (there ? r : 0), n = f / p.G, h = u.h * p.G + f - n * p.G;
        copy16(q_at + (r >> 7) * W::kEntry + place(r & 127, piece),
               p.q + u.b * p.q_seq + n * p.q_token + h * p.q_head + piece * 16, there);
      }
      copy_commit();
      copy_wait<0>();
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive(&ctl.q_full);
      if constexpr (NQ == 2) {
        for (int i = 1; ok && i < n_tiles; ++i) {
          copy_entry(false, i);
          if (ok) copy_entry(true, i);
        }
      } else {
        for (int i = 0; ok && i < n_tiles; ++i) {
          copy_entry(true, i);
          if (ok && i + 2 < n_tiles) copy_entry(false, i + 2);
        }
      }
      if (!ok) break;
      tiles_before += n_tiles;
      w += n_tiles;
      if (w >= line.w1) break;
      u.next(p, line);
    }
    if (ok) flush();
    copy_wait<0>();
  } else if (lane == 0) {
    // ------------------------------------------------------------- products
    const uint32_t ring_at = smem_u32(ring), q_at = smem_u32(q_s);
    constexpr uint32_t s_idesc = mma_idesc<E>(kTileKeys, false), o_idesc = mma_idesc<E>(D, true);
    uint32_t taken = 0, n_p[2] = {0, 0}, n_q = 0;
    bool ok = true;
    // Waits for the next entry of the ring; its place.
    auto take = [&]() {
      const int slot = taken % W::kRing;
      ok = bar_wait(&ctl.full[slot], (taken / W::kRing) & 1u, &ctl.dead);
      ++taken;
      return slot;
    };
    auto scores = [&](int g, int slot) {
      const uint32_t a = q_at + (NQ == 2 ? g * W::kEntry : 0), b = ring_at + slot * W::kEntry;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = (k >> 2) * W::kPanel + (k & 3) * 32;
        mma_ss(tmem + g * 128, smem_desc(a + off, 16, 1024), smem_desc(b + off, 16, 1024), s_idesc,
               k > 0);
      }
      mma_commit(&ctl.s_full[g]);
    };
    auto outputs = [&](int g, int slot, bool first) {
      ok = bar_wait(&ctl.p_full[g], n_p[g]++ & 1u, &ctl.dead);
      if (!ok) return;
      tc_after();
      const uint32_t b = ring_at + slot * W::kEntry;
#pragma unroll
      for (int k = 0; k < kTileKeys / 16; ++k)
        mma_ts(tmem + 256 + g * 128, tmem + g * 128 + k * 8,
               smem_desc(b + k * 16 * W::kRow, W::kPanel, 1024), o_idesc, !first || k > 0);
    };
    for (long long w = line.w0; ok;) {
      const int n_tiles = u.i1 - u.i0, live = u.live_rows(p);
      if constexpr (NQ == 2) {
        const int streams = live > 128 ? 2 : 1;
        int key_slot = take();
        if (!ok || !(ok = bar_wait(&ctl.q_full, n_q++ & 1u, &ctl.dead))) break;
        for (int g = 0; g < streams; ++g) scores(g, key_slot);
        mma_commit(&ctl.empty[key_slot]);
        if (n_tiles == 1) mma_commit(&ctl.q_empty);
        for (int i = 0; i < n_tiles; ++i) {
          const int val_slot = take();
          if (!ok) break;
          const bool more = i + 1 < n_tiles;
          for (int g = 0; g < streams; ++g) {
            outputs(g, val_slot, i == 0);
            if (!ok) break;
            if (!more) mma_commit(&ctl.o_done[g]);
            if (g == streams - 1) mma_commit(&ctl.empty[val_slot]);
            if (more) {
              if (g == 0) key_slot = take();
              if (!ok) break;
              scores(g, key_slot);
              if (g == streams - 1) {
                mma_commit(&ctl.empty[key_slot]);
                if (i + 2 == n_tiles) mma_commit(&ctl.q_empty);
              }
            }
          }
          if (!ok) break;
        }
      } else {
        int slot = take();
        if (!ok || !(ok = bar_wait(&ctl.q_full, n_q++ & 1u, &ctl.dead))) break;
        scores(0, slot);
        mma_commit(&ctl.empty[slot]);
        if (n_tiles > 1) {
          slot = take();
          if (!ok) break;
          scores(1, slot);
          mma_commit(&ctl.empty[slot]);
        }
        if (n_tiles <= 2) mma_commit(&ctl.q_empty);
        for (int i = 0; i < n_tiles; ++i) {
          const int g = i & 1;
          slot = take();
          if (!ok) break;
          outputs(g, slot, i < 2);
          if (!ok) break;
          mma_commit(&ctl.empty[slot]);
          if (i + 2 >= n_tiles) mma_commit(&ctl.o_done[g]);
          if (i + 2 < n_tiles) {
            slot = take();
            if (!ok) break;
            scores(g, slot);
            mma_commit(&ctl.empty[slot]);
            if (i + 3 == n_tiles) mma_commit(&ctl.q_empty);
          }
        }
      }
      if (!ok) break;
      w += n_tiles;
      if (w >= line.w1) break;
      u.next(p, line);
    }
    // nothing is in flight when the tensor memory goes back
    mma_commit(&ctl.drain);
    const uint32_t drain = smem_u32(&ctl.drain);
    for (const long long t0 = clock64(); !bar_test(drain, 0u) && clock64() - t0 < kWaitCycles;) {
    }
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 12)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  if (tid == 0 && ctl.dead && p.flags) {
    // a wait gave up: the outputs of the run's sequences are not to be used
    UnitWalk v;
    v.start(p, line);
    for (long long w = line.w0;;) {
      atomicOr(p.flags + v.b, SPEC_FLAG_TIMEOUT);
      w += v.i1 - v.i0;
      if (w >= line.w1) break;
      v.next(p, line);
    }
  }
}

template <class E, int D, int NQ>
cudaError_t start_wide(const AttnParams &p, cudaStream_t stream) {
  constexpr int smem = wide_smem<D, NQ>();
  const cudaError_t e = cudaFuncSetAttribute(wide_kernel<E, D, NQ>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  wide_kernel<E, D, NQ><<<p.ctas, kWideThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <class E>
cudaError_t start_wide(const AttnParams &p, cudaStream_t stream) {
  if (p.D == 64)
    return p.rows == 256 ? start_wide<E, 64, 2>(p, stream) : start_wide<E, 64, 1>(p, stream);
  return p.rows == 256 ? start_wide<E, 128, 2>(p, stream) : start_wide<E, 128, 1>(p, stream);
}

cudaError_t launch_attention_wide(const AttnParams &p, int dtype, cudaStream_t stream) {
  return dtype == SPEC_BF16 ? start_wide<Bf16>(p, stream) : start_wide<F16>(p, stream);
}

}  // namespace sv
