// Attention over a paged cache on the fifth-generation tensor cores: 16-bit
// types, head_dim 64 or 128, pages of 8, 16, 32, 64 or a multiple of 128 tokens,
// units of 128 or 256 rows (new tokens times the query heads of a group).
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
// Warps 0-3 and 4-7: the softmax of stream 0 and 1; warps without rows only
// pass their barriers, so few rows cost few instructions.  Warps 8 and 9: keys
// and values by TMA, one box per page, into a ring of entries of 128 rows; warp
// 10: the queries' boxes.  One thread of warp 11 issues every product.  Copies
// and products meet at mbarriers; every wait is bounded.
//
// Shared rows are 128-byte pieces in the 128-byte swizzle.  An entry of keys or
// values is groups of eight tokens, each with its panels of 64 elements one
// behind another, so that one box holds a page whole whatever its size; rows of
// K are K-major for S = Q K^T, rows of V are N-major for O += P V, without a
// transpose.  A tile of queries is its panels one behind another, rows token by
// token with the group's heads, as many whole tokens as 128 rows hold.
//
// One token is bound by HBM: 64 KB of keys and values a tile at head_dim 128
// arrive in about 3000 cycles of an SM, their products take 512 of them.
#include <climits>
#include <numeric>

#include "paged_attention.cuh"

namespace sv {

namespace {

constexpr int kSoft = 256;          // softmax threads
constexpr int kWideThreads = 384;   // three warpgroups
// Registers of a softmax thread and of the others: 2 * 128 * 208 + 128 * 88 are
// the 384 * 168 that the CTA is launched with.
constexpr int kSoftRegs = 208, kRestRegs = 88;
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
  static constexpr int kPanels = D / 64;
  static constexpr int kPanel = 8 * kRow;             // 8 rows of 64 elements
  static constexpr int kGroup = kPanels * kPanel;     // 8 rows
  static constexpr int kEntry = kTileKeys / 8 * kGroup;
  static constexpr int kQPanel = 128 * kRow;          // of queries: 128 rows
  // queries of 256 rows, or of this unit and the next
  static constexpr int kQ = 2 * kEntry;
  static constexpr int kRing = D == 128 ? 5 : 12;  // what 227 KB hold beside them
};

template <int D, int NQ>
struct WideCtl {
  using W = WideShape<D, NQ>;
  unsigned long long full[W::kRing], empty[W::kRing], s_full[2], p_full[2], o_done[2], q_full[2],
      q_empty[2], meet, drain;
  long long warp_s[kWideThreads / 32], found_s[2];
  alignas(16) uint32_t valid[kValidRing][4];
  uint32_t tmem;
  int dead, bad;
  float ml[NQ == 1 ? 2 : 1][2][NQ == 1 ? 128 : 1];
};

template <int D, int NQ>
constexpr int wide_smem() {
  return WideShape<D, NQ>::kQ + WideShape<D, NQ>::kRing * WideShape<D, NQ>::kEntry +
         static_cast<int>(sizeof(WideCtl<D, NQ>));
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

// A last wait, whether others have given up or not.
__device__ __forceinline__ void bar_linger(const void *bar, uint32_t parity) {
  const uint32_t at = smem_u32(bar);
  for (const long long t0 = clock64(); !bar_test(at, parity) && clock64() - t0 < kWaitCycles / 16;) {
  }
}
// bar_wait by a whole warp, which goes on together.
__device__ __forceinline__ bool warp_wait(const void *bar, uint32_t parity, int *dead) {
  return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, dead));
}

__device__ __forceinline__ void bar_expect(const void *bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void box_load(uint32_t to, const CUtensorMap *map, const void *bar, int x0,
                                         int x1, int x2, int x3, int x4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(to),
      "l"(map), "r"(smem_u32(bar)), "r"(x0), "r"(x1), "r"(x2), "r"(x3), "r"(x4)
      : "memory");
}
template <int kRegs>
__device__ __forceinline__ void more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
// Two float32 operations at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long &>(d))
      : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)),
        "l"(reinterpret_cast<unsigned long long &>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long &>(d))
      : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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
__device__ __forceinline__ void tm_load16(uint32_t (&r)[16], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(at)
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

// Place in the order of a unit's entries, with 128 rows, of the values of its
// tile i of n: K0 K1 V0 K2 V1 K3 ... V(n-2) V(n-1); the keys of tile i > 0 are
// at 2 i - 1.  With 256 rows the order is K0 V0 K1 V1 ...
__device__ __forceinline__ int value_entry(int i, int n) { return i + 1 < n ? 2 * i + 2 : 2 * i + 1; }

// The top bit of each of two 16-bit values that is an infinity or a NaN.
template <class E>
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t v) {
  constexpr uint32_t exps = E::kExp * 0x10001u, ones = (E::kExp & (0u - E::kExp)) * 0x10001u;
  return ((v & exps) + ones) & 0x80008000u;
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
__global__ void __launch_bounds__(kWideThreads, 1)
    wide_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ WideMaps maps) {
  using W = WideShape<D, NQ>;
  using Ctl = WideCtl<D, NQ>;
  using TE = typename E::T;
  // all shared memory is this array, so its alignment is the swizzle's
  extern __shared__ __align__(1024) char wide_s[];
  char *q_s = wide_s, *ring = wide_s + W::kQ;
  Ctl &ctl = *reinterpret_cast<Ctl *>(ring + W::kRing * W::kEntry);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);

  if (tid == 0) {
    for (int i = 0; i < W::kRing; ++i) {
      bar_init(&ctl.full[i], 1);
      bar_init(&ctl.empty[i], 1);
    }
    for (int g = 0; g < 2; ++g) {
      bar_init(&ctl.s_full[g], 1);
      bar_init(&ctl.p_full[g], 4);
      bar_init(&ctl.o_done[g], 1);
      bar_init(&ctl.q_full[g], 1);
      bar_init(&ctl.q_empty[g], 1);
    }
    bar_init(&ctl.meet, kSoft / 32);
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
  if (warp == 11) {
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
    more_regs<kSoftRegs>();
    const int g = warp >> 2;
    const int lane_row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + g * 128, o_at = tmem + lanes + 256;
    const float c = p.scale_log2;
    const int tile_rows = NQ == 2 ? p.rows / 2 : p.rows;
    uint32_t n_s = 0, n_o[2] = {0, 0}, n_meet = 0;
    int tiles_before = 0;  // of this CTA, for the rings
    bool ok = true;
    for (long long w = line.w0; ok;) {
      const int n_tiles = u.i1 - u.i0, live = u.live_rows(p);
      const int row = NQ == 2 ? g * tile_rows + lane_row : lane_row;
      const int rows = NQ == 2 ? min(tile_rows, live - g * tile_rows) : live;  // of the stream
      const bool mine = lane_row < rows;
      const int n = (u.r0 + min(row, live - 1)) / p.G;
      const bool active = rows > 0;
      const bool works = (lane_row & ~31) < rows;  // this warp has rows
      float m = -INFINITY, l = 0.f;
      for (int i = NQ == 2 ? 0 : g; active && i < n_tiles; i += NQ == 2 ? 1 : 2) {
        if (!(ok = warp_wait(&ctl.s_full[g], n_s++ & 1u, &ctl.dead))) break;
        const int at0 = key_tile(u.k, u.i0 + i) * kTileKeys;
        const uint4 valid =
            *reinterpret_cast<const uint4 *>(ctl.valid[(tiles_before + i) % kValidRing]);
        const bool masked = (valid.x & valid.y & valid.z & valid.w) != 0xFFFFFFFFu ||
                            !all_seen(p, u.k, u.r0, at0, kTileKeys);
        if (works) {
          tc_after();
          uint32_t s[4][32];
#pragma unroll
          for (int j = 0; j < 4; ++j) tm_load32(s[j], s_at + j * 32);
          tm_wait_ld();
          if (masked) {
            const uint32_t in[4] = {valid.x, valid.y, valid.z, valid.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t vis = seen_word(p, u.k, u.b, n, at0 + j * 32, in[j]);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((vis >> e) & 1u)) s[j][e] = __float_as_uint(-INFINITY);
            }
          }
          float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              x[j] = max3(x[j], __uint_as_float(s[j][e]), __uint_as_float(s[j][e + 1]));
          const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * c;
          const bool raise = mine && top > m + kSlack;
          if (__any_sync(0xFFFFFFFFu, raise)) {
            const float to = raise ? top : m;
            const float f = m == -INFINITY ? 0.f : fast_exp2(m - to);
            l *= f;
            m = to;
            if (i >= (NQ == 2 ? 1 : 2)) {
              // the products before S's are complete: O is whole
#pragma unroll 1
              for (int d = 0; d < D; d += 16) {
                uint32_t o[16];
                tm_load16(o, o_at + g * 128 + d);
                tm_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tm_store16(o_at + g * 128 + d, o);
              }
            }
          }
          const float sub = m == -INFINITY ? 0.f : -m;
          const float2 c2 = make_float2(c, c), sub2 = make_float2(sub, sub);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t packed[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float2 y = fma2(make_float2(__uint_as_float(s[j][e]), __uint_as_float(s[j][e + 1])), c2,
                              sub2);
              y.x = fast_exp2(y.x);
              y.y = fast_exp2(y.y);
              sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], y);
              // the product takes the weights in the cache's type: each is off
              // by at most half a step of that type, as the values themselves are
              packed[e / 2] = E::pack(y.x, y.y);
            }
            tm_store16(s_at + j * 16, packed);
          }
          sum[0] = add2(sum[0], sum[1]);
          l += sum[0].x + sum[0].y;
          tm_wait_st();
        }
        if (masked && (NQ == 1 || g == 0)) {
          // Rows of the value tile that some row of the unit does not see: those
          // that were not copied become zero, and so do infinities and NaNs,
          // which nonfinite_values adds to the rows that see them.  With 256 rows
          // the first stream does it, whose product with the tile comes first.
          const int e = NQ == 2 ? 2 * (tiles_before + i) + 1 : 2 * tiles_before + value_entry(i, n_tiles);
          const int slot = e % W::kRing;
          if (!(ok = warp_wait(&ctl.full[slot], (e / W::kRing) & 1, &ctl.dead))) break;
          bool found = false;
          char *at = ring + slot * W::kEntry + lane_row * 16;
          const int key0 = (lane_row * 16 / W::kGroup) * 8 + lane_row / 8 % 8;
#pragma unroll 4
          for (int t = 0; t < W::kEntry / 2048; ++t) {
            const int key = key0 + t * 2048 / W::kGroup * 8;
            uint4 *x = reinterpret_cast<uint4 *>(at + t * 2048);
            const uint4 y = *x;
            const uint32_t word = key < 64 ? (key < 32 ? valid.x : valid.y)
                                           : (key < 96 ? valid.z : valid.w);
            if (!((word >> (key & 31)) & 1u)) {
              *x = make_uint4(0, 0, 0, 0);
            } else if (nonfinite_bits<E>(y.x) | nonfinite_bits<E>(y.y) | nonfinite_bits<E>(y.z) |
                       nonfinite_bits<E>(y.w)) {
              *x = make_uint4(finite_or_zero<E>(y.x), finite_or_zero<E>(y.y), finite_or_zero<E>(y.z),
                              finite_or_zero<E>(y.w));
              found = true;
            }
          }
          if (found) *reinterpret_cast<volatile int *>(&ctl.bad) = 1;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&ctl.p_full[g]);
      }
      if (!ok) break;
      tiles_before += n_tiles;

      // the unit's end
      const bool whole = u.whole();
      float *slot = p.part + piece_slot(u) * slot_floats(p.rows, D);
      const long long out_at = mine ? out_row(p, u.b, u.h, u.r0 + row) : 0;
      const int d_from = NQ == 2 ? 0 : g * (D / 2), d_to = NQ == 2 ? D : d_from + D / 2;
      float w0 = 1.f, w1 = 0.f;  // weights of the streams' outputs
      if constexpr (NQ == 2) {
        if (active && !(ok = warp_wait(&ctl.o_done[g], n_o[g]++ & 1u, &ctl.dead))) break;
      } else {
        ctl.ml[g][0][lane_row] = m;
        ctl.ml[g][1][lane_row] = l;
        __syncwarp();
        if (lane == 0) bar_arrive(&ctl.meet);
        if (!(ok = warp_wait(&ctl.meet, n_meet++ & 1u, &ctl.dead))) break;
        if (!(ok = warp_wait(&ctl.o_done[0], n_o[0]++ & 1u, &ctl.dead))) break;
        if (n_tiles > 1 && !(ok = warp_wait(&ctl.o_done[1], n_o[1]++ & 1u, &ctl.dead))) break;
        const float m0 = ctl.ml[0][0][lane_row], m1 = ctl.ml[1][0][lane_row];
        m = fmaxf(m0, m1);
        w0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - m);
        w1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - m);
        l = (w0 == 0.f ? 0.f : w0 * ctl.ml[0][1][lane_row]) +
            (w1 == 0.f ? 0.f : w1 * ctl.ml[1][1][lane_row]);
      }
      if (active && works) {
        tc_after();
        const float norm = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        const bool bad = *reinterpret_cast<volatile int *>(&ctl.bad) != 0;
#pragma unroll 1
        for (int d = d_from; d < d_to; d += 32) {
          __syncwarp();
          uint32_t o[32];
          tm_load32(o, o_at + (NQ == 2 ? g * 128 : 0) + d);
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
          } else {
            tm_wait_ld();
          }
          if (mine) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float4 v = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                     __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
              if (l == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
              if (whole) {
                v = make_float4(v.x * norm, v.y * norm, v.z * norm, v.w * norm);
                store4(static_cast<TE *>(p.out) + out_at * D + d + e, v);
              } else {
                store4(slot + 2 * p.rows + static_cast<size_t>(row) * D + d + e, v);
              }
            }
          }
        }
        if (bad && mine && l != 0.f) {
          for (int d = d_from; d < d_to; d += 4) {
            const float4 v =
                nonfinite_values<TE, kTileKeys>(p, u, n, d, make_float4(0.f, 0.f, 0.f, 0.f));
            const float x[4] = {v.x, v.y, v.z, v.w};
            for (int e = 0; e < 4; ++e) {
              if (x[e] == 0.f) continue;
              if (whole) {
                TE *o = static_cast<TE *>(p.out) + out_at * D + d + e;
                *o = E::from(E::to(*o) + x[e]);
              } else {
                slot[2 * p.rows + static_cast<size_t>(row) * D + d + e] += x[e];
              }
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
      }
      __syncwarp();
      tc_before();
      if constexpr (NQ == 1) {
        // both halves have been read before either stream's next output begins
        if (lane == 0) bar_arrive(&ctl.meet);
        if (!(ok = warp_wait(&ctl.meet, n_meet++ & 1u, &ctl.dead))) break;
      }
      w += n_tiles;
      if (w >= line.w1) break;
      u.next(p, line);
    }
  } else {
    fewer_regs<kRestRegs>();
    if (warp < 10) {
      // ----------------------------------------------------- keys and values
      const bool values = warp == 9;
      const CUtensorMap *map = values ? &maps.v : &maps.k;
      const int unit_page = values ? maps.v_page : maps.k_page;
      const int unit_head = values ? maps.v_head : maps.k_head;
      const int unit_token = values ? maps.v_token : maps.k_token;
      const uint32_t ring_at = smem_u32(ring);
      const int box = min(p.C.page_size, kTileKeys);  // tokens of a box
      const int boxes = kTileKeys / box;              // of a tile, one per lane
      const uint32_t all = low_bits(boxes);
      const int shift = 31 - __clz(box);
      uint32_t last = 0;
      int tiles_before = 0;
      bool ok = true;
      auto look_up = [&](int i) {  // this lane's page of tile i of the unit
        const int at = key_tile(u.k, u.i0 + i) * kTileKeys + lane * box;
        if (lane >= boxes || i >= u.i1 - u.i0 || at >= u.k.end) return -1;
        return page_at(p.S, u.b, p.C.page_size <= kTileKeys ? at >> shift : at / p.C.page_size);
      };
      for (long long w = line.w0; ok;) {
        const int n_tiles = u.i1 - u.i0;
        // a tile's pages are looked up two tiles ahead
        int page = look_up(0), next = look_up(1);
        for (int i = 0; i < n_tiles; ++i) {
          const int behind = look_up(i + 2);
          const uint32_t e =
              2 * tiles_before + (NQ == 2 ? 2 * i + (values ? 1 : 0)
                                          : (values ? value_entry(i, n_tiles) : max(2 * i - 1, 0)));
          const int slot = e % W::kRing;
          if (!(ok = warp_wait(&ctl.empty[slot], ((e / W::kRing) & 1u) ^ 1u, &ctl.dead))) break;
          const bool there = page_ok(p.C, page);
          const uint32_t pages = __ballot_sync(0xFFFFFFFFu, there);
          const int at0 = key_tile(u.k, u.i0 + i) * kTileKeys;
          if (!values && lane < 4) {
            uint32_t word = 0xFFFFFFFFu;
            if (pages != all || at0 + kTileKeys > u.k.end) {
              word = 0u;
              for (int k = 0; k < 32; k += box)
                if ((pages >> ((lane * 32 + k) >> shift)) & 1u) word |= low_bits(box) << k;
              word &= low_bits(u.k.end - at0 - lane * 32);
            }
            ctl.valid[(tiles_before + i) % kValidRing][lane] = word;
          }
          __syncwarp();
          if (lane == 0) bar_expect(&ctl.full[slot], __popc(pages) * box * W::kRow * W::kPanels);
          __syncwarp();
          if (there) {
            const int token = p.C.page_size <= kTileKeys ? 0 : at0 % p.C.page_size;
            box_load(ring_at + slot * W::kEntry + lane * (box >> 3) * W::kGroup, map,
                     &ctl.full[slot], 0, 0, 0, 0, page * unit_page + u.h * unit_head + token * unit_token);
          }
          last = e;
          page = next;
          next = behind;
        }
        if (!ok) break;
        tiles_before += n_tiles;
        w += n_tiles;
        if (w >= line.w1) break;
        u.next(p, line);
      }
      // the products wait for every entry; where a wait gave up, its copies are
      // given time to land before the CTA ends
      for (uint32_t e = last + 1 > W::kRing ? last + 1 - W::kRing : 0; !ok && e <= last; ++e)
        bar_linger(&ctl.full[e % W::kRing], (e / W::kRing) & 1u);
    } else if (warp == 10) {
      // -------------------------------------------------------------- queries
      const uint32_t q_at = smem_u32(q_s);
      const int tile_rows = NQ == 2 ? p.rows / 2 : p.rows;
      uint32_t unit = 0;
      bool ok = true;
      for (long long w = line.w0;;) {
        const int live = u.live_rows(p);
        const int buf = NQ == 1 ? unit & 1 : 0;
        const uint32_t use = NQ == 1 ? unit >> 1 : unit;
        // once the products of the unit before have read theirs
        if (!(ok = warp_wait(&ctl.q_empty[buf], (use & 1u) ^ 1u, &ctl.dead))) break;
        if (lane == 0) {
          const int tiles = NQ == 2 && live > tile_rows ? 2 : 1;
          bar_expect(&ctl.q_full[buf], tiles * tile_rows * W::kRow * W::kPanels);
          for (int t = 0; t < tiles; ++t)
            for (int x = 0; x < W::kPanels; ++x)
              box_load(q_at + (buf + t) * W::kEntry + x * W::kQPanel, &maps.q, &ctl.q_full[buf], 0, 0,
                       (u.r0 + t * tile_rows) / p.G, x, u.b * maps.q_seq + u.h * maps.q_head);
        }
        __syncwarp();
        ++unit;
        w += u.i1 - u.i0;
        if (w >= line.w1) break;
        u.next(p, line);
      }
      for (int b = 0; !ok && b < 2; ++b) {
        const uint32_t uses = NQ == 1 ? (unit + 1 - b) / 2 : (b == 0 ? unit : 0);
        if (uses > 0) bar_linger(&ctl.q_full[b], (uses - 1) & 1u);
      }
    } else if (lane == 0) {
      // ------------------------------------------------------------- products
      const uint32_t ring_at = smem_u32(ring), q_at = smem_u32(q_s);
      constexpr uint32_t s_idesc = mma_idesc<E>(kTileKeys, false), o_idesc = mma_idesc<E>(D, true);
      uint32_t taken = 0, n_p[2] = {0, 0}, unit = 0;
      bool ok = true;
      // Waits for the next entry of the ring; its place.
      auto take = [&]() {
        const int slot = taken % W::kRing;
        ok = bar_wait(&ctl.full[slot], (taken / W::kRing) & 1u, &ctl.dead);
        ++taken;
        return slot;
      };
      auto scores = [&](int g, int buf, int slot) {
        // a descriptor's address counts 16 bytes
        const uint64_t a = smem_desc(q_at + buf * W::kEntry, 16, 1024);
        const uint64_t b = smem_desc(ring_at + slot * W::kEntry, 16, W::kGroup);
        tc_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss(tmem + g * 128, a + ((k >> 2) * W::kQPanel + (k & 3) * 32) / 16,
                 b + ((k >> 2) * W::kPanel + (k & 3) * 32) / 16, s_idesc, k > 0);
        mma_commit(&ctl.s_full[g]);
      };
      auto outputs = [&](int g, int slot, bool first) {
        ok = bar_wait(&ctl.p_full[g], n_p[g]++ & 1u, &ctl.dead);
        if (!ok) return;
        tc_after();
        const uint64_t b = smem_desc(ring_at + slot * W::kEntry, W::kPanel, W::kGroup);
#pragma unroll
        for (int k = 0; k < kTileKeys / 16; ++k)
          mma_ts(tmem + 256 + g * 128, tmem + g * 128 + k * 8, b + k * 2 * W::kGroup / 16, o_idesc,
                 !first || k > 0);
      };
      for (long long w = line.w0; ok;) {
        const int n_tiles = u.i1 - u.i0, live = u.live_rows(p);
        const int buf = NQ == 1 ? unit & 1 : 0;
        const uint32_t use = NQ == 1 ? unit >> 1 : unit;
        int slot = take();
        if (!ok || !(ok = bar_wait(&ctl.q_full[buf], use & 1u, &ctl.dead))) break;
        ++unit;
        if constexpr (NQ == 2) {
          const int streams = live > p.rows / 2 ? 2 : 1;
          for (int g = 0; g < streams; ++g) scores(g, g, slot);
          mma_commit(&ctl.empty[slot]);
          if (n_tiles == 1) mma_commit(&ctl.q_empty[0]);
          for (int i = 0; ok && i < n_tiles; ++i) {
            const int val_slot = take();
            if (!ok) break;
            const bool more = i + 1 < n_tiles;
            for (int g = 0; g < streams; ++g) {
              outputs(g, val_slot, i == 0);
              if (!ok) break;
              if (!more) mma_commit(&ctl.o_done[g]);
              if (g == streams - 1) mma_commit(&ctl.empty[val_slot]);
              if (more) {
                if (g == 0) slot = take();
                if (!ok) break;
                scores(g, g, slot);
                if (g == streams - 1) {
                  mma_commit(&ctl.empty[slot]);
                  if (i + 2 == n_tiles) mma_commit(&ctl.q_empty[0]);
                }
              }
            }
          }
        } else {
          scores(0, buf, slot);
          mma_commit(&ctl.empty[slot]);
          if (n_tiles > 1) {
            slot = take();
            if (!ok) break;
            scores(1, buf, slot);
            mma_commit(&ctl.empty[slot]);
          }
          if (n_tiles <= 2) mma_commit(&ctl.q_empty[buf]);
          for (int i = 0; ok && i < n_tiles; ++i) {
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
              scores(g, buf, slot);
              mma_commit(&ctl.empty[slot]);
              if (i + 3 == n_tiles) mma_commit(&ctl.q_empty[buf]);
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
      bar_linger(&ctl.drain, 0u);
    }
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 11)
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

namespace {

// cuTensorMapEncodeTiled of the installed driver; the library does not link to it.
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled found = [] {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult status;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &status) != cudaSuccess ||
        status != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiled>(nullptr);
    return reinterpret_cast<EncodeTiled>(fn);
  }();
  return found;
}

bool encode_map(CUtensorMap *map, int dtype, const char *base, const cuuint64_t (&dims)[5],
                const long long (&strides)[4], const cuuint32_t (&box)[5]) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  cuuint64_t bytes[4];
  for (int i = 0; i < 4; ++i) bytes[i] = static_cast<cuuint64_t>(strides[i]);
  return encode(map,
                dtype == SPEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                5, const_cast<char *>(base), dims, bytes, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The fifth dimension of the maps counts the largest step that the other
// strides (of pages, heads and tokens; of sequences and heads) are multiples of,
// so that one coordinate says where a box begins.
struct Origin {
  long long step, count;
  int units[3];
};
bool origin(Origin *o, const long long (&strides)[3], const long long (&sizes)[3]) {
  long long step = 0;
  for (int i = 0; i < 3; ++i)
    if (sizes[i] > 1) step = std::gcd(step, strides[i]);
  o->step = step == 0 ? 16 : step;
  o->count = 1;
  for (int i = 0; i < 3; ++i) {
    const long long units = sizes[i] > 1 ? strides[i] / o->step : 0;
    if (units > INT_MAX / sizes[i]) return false;
    o->units[i] = static_cast<int>(units);
    o->count += units * (sizes[i] - 1);
  }
  return o->count <= INT_MAX;
}

// One layer's keys or values: [64 elements, 8 tokens, panels, groups of 8
// tokens, origin]; a box is the tokens of a page, at most 128.
bool cache_map(CUtensorMap *map, Origin *o, int dtype, const KvCache &C, int D, const char *base,
               long long page, long long token, long long head) {
  const long long strides[3] = {page, head, token};
  const long long sizes[3] = {C.pages, C.heads, C.page_size > kTileKeys ? C.page_size : 1};
  if (!origin(o, strides, sizes)) return false;
  const int box_tokens = C.page_size < kTileKeys ? C.page_size : kTileKeys;
  const cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(D / 64),
                              static_cast<cuuint64_t>(box_tokens / 8),
                              static_cast<cuuint64_t>(o->count)};
  const long long steps[4] = {token, 128, 8 * token, o->step};
  const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(D / 64),
                             static_cast<cuuint32_t>(box_tokens / 8), 1};
  return encode_map(map, dtype, base, dims, steps, box);
}

template <class E, int D, int NQ>
cudaError_t start_wide(const AttnParams &p, const WideMaps &maps, cudaStream_t stream) {
  constexpr int smem = wide_smem<D, NQ>();
  const cudaError_t e = cudaFuncSetAttribute(wide_kernel<E, D, NQ>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  wide_kernel<E, D, NQ><<<p.ctas, kWideThreads, smem, stream>>>(p, maps);
  return cudaGetLastError();
}

template <class E>
cudaError_t start_wide(const AttnParams &p, int tiles, const WideMaps &maps, cudaStream_t stream) {
  if (p.D == 64) return tiles == 2 ? start_wide<E, 64, 2>(p, maps, stream) : start_wide<E, 64, 1>(p, maps, stream);
  return tiles == 2 ? start_wide<E, 128, 2>(p, maps, stream) : start_wide<E, 128, 1>(p, maps, stream);
}

}  // namespace

bool wide_maps(const AttnParams &p, int dtype, WideMaps *maps) {
  Origin k, v, q;
  if (!cache_map(&maps->k, &k, dtype, p.C, p.D, p.C.k, p.C.k_page, p.C.k_token, p.C.k_head) ||
      !cache_map(&maps->v, &v, dtype, p.C, p.D, p.C.v, p.C.v_page, p.C.v_token, p.C.v_head))
    return false;
  maps->k_page = k.units[0];
  maps->k_head = k.units[1];
  maps->k_token = k.units[2];
  maps->v_page = v.units[0];
  maps->v_head = v.units[1];
  maps->v_token = v.units[2];
  // queries: [64 elements, heads of a group, tokens, panels, origin]; a box is
  // the rows of a tile in one panel, zero behind the last token
  const long long row = static_cast<long long>(p.D) * 2;
  const long long strides[3] = {p.q_seq, p.G * p.q_head, 0}, sizes[3] = {p.S.B, p.C.heads, 1};
  if (!origin(&q, strides, sizes)) return false;
  maps->q_seq = q.units[0];
  maps->q_head = q.units[1];
  const cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(p.G), static_cast<cuuint64_t>(p.S.N),
                              static_cast<cuuint64_t>(p.D / 64), static_cast<cuuint64_t>(q.count)};
  const long long steps[4] = {p.G > 1 ? p.q_head : row, p.S.N > 1 ? p.q_token : row, 128, q.step};
  const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(p.G),
                             static_cast<cuuint32_t>(wide_tile_rows(p.G) / p.G), 1, 1};
  return encode_map(&maps->q, dtype, p.q, dims, steps, box);
}

cudaError_t launch_attention_wide(const AttnParams &p, int tiles, const WideMaps &maps, int dtype,
                                  cudaStream_t stream) {
  return dtype == SPEC_BF16 ? start_wide<Bf16>(p, tiles, maps, stream)
                            : start_wide<F16>(p, tiles, maps, stream);
}

}  // namespace sv
