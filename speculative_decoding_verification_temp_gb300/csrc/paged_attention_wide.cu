// Attention over a paged cache on the fifth-generation tensor cores: 16-bit
// types, head_dim 64 or 128, pages of a multiple of 8 tokens,
// rows in tiles of at most 128 (new tokens times the query heads of a group).
//
// For a tile of 128 keys a stream of work computes S = Q K^T into tensor memory
// (128 lanes of rows x 128 columns); one thread per row turns S into weights in
// place (the running maximum, the sum, 2^(s c - m) packed into the first half of
// S's columns), and O += P V takes them from there as the A operand.  Two
// streams share a CTA, so that the products of one run while the other is in its
// softmax:
//   solo_kernel  units of one row tile; each stream has units, keys and values
//                of its own.  Up to 32 rows are given to each of the four
//                quarters of the lanes, and each quarter weighs a quarter of a
//                tile's keys: a row's softmax is four threads' work, and the
//                quarters' results are added at the unit's end.
//   pair_kernel  units of two row tiles, one per stream, that share the keys and
//                values
//
// Keys and values come by TMA, one box per page or part of one, into a ring of
// entries of 128 rows; every hand-over is an mbarrier, every wait is bounded.  Shared rows are
// 128-byte pieces in the 128-byte swizzle.  An entry of keys or values is groups
// of eight tokens, each with its panels of 64 elements one behind another, so
// that one box holds a page whole whatever its size; rows of K are K-major for
// S = Q K^T, rows of V are N-major for O += P V, without a transpose.  A tile of
// queries is its panels one behind another, rows token by token with the
// group's heads, as many whole tokens as 128 rows hold.
//
// One token is bound by HBM: 64 KB of keys and values a tile at head_dim 128
// arrive in about 3000 cycles of an SM; a stream's tile takes 1024 of products (64 a
// step of 16 in Q K^T and P V alike, the pipe's rate: from the share of the time that
// the pipe is active) and 600 of softmax in quarters.  256 sequences of 1 to 4096 tokens, one token each, 32 query
// heads on 8 of 128 bf16: 333 us, 6.48 TB/s, 0.95 of the measured copy rate, DRAM
// reads 1.004 of the keys' and values' bytes.
//
// Many rows are bound by the turns that a stream's softmax (1770 cycles a tile
// with both streams at it) and products take with one buffer of scores: scores, all
// their weights, outputs, one after the other.  256-node trees at B = 16, 64 query
// heads on 8 of 128 bf16, contexts of 1000 to 8192 tokens: 519 to 530 us, 1.16
// PFLOP/s; a pair of tiles takes about 3900 cycles, of which its products need 2048.
// Measured and not kept: against 530 us waits that suspend (566 us) or only poll (566)
// and ends of units stored by quads in whole lines (554); against 645 us, before row
// tiles had lines of their own, and not measured since: scores in halves of 64 keys
// with two buffers (710 us, 2520 cycles of products a tile) and two warps per row
// (671).
#include <climits>
#include <numeric>

#include "paged_attention.cuh"

namespace sv {

namespace {

constexpr int kWideThreads = 384;  // three warpgroups
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
// How far float16 weights are lifted: m lies so far below the maximum that it was
// raised to, so that weights reach 2^(kLift + kSlack) = 2^15 at most, and those that
// float16 rounds to zero are below 2^-32 of the row's largest instead of 2^-25.
constexpr float kLift = 7.f;

// Bytes of an entry of 128 rows.
template <int D>
struct Entry {
  static constexpr int kRow = 128;              // of a row in a panel
  static constexpr int kPanels = D / 64;
  static constexpr int kPanel = 8 * kRow;       // 8 rows of 64 elements
  static constexpr int kGroup = kPanels * kPanel;
  static constexpr int kBytes = kTileKeys / 8 * kGroup;
};

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

// The first wait of a run, for the keys of its first tile, where a caller has
// shortened it (limit <= 0: one non-blocking test); by one warp, the others find in
// their own waits that it gave up.  (In pair_kernel the warp that checks values: before
// the products' loop it costs 256-node trees 1 % of their time.)
__device__ __forceinline__ void first_wait(const void *bar, long long limit, int *dead) {
  if (limit >= kWaitCycles) return;
  const uint32_t at = smem_u32(bar);
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], 0;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(at)
      : "memory");
  for (const long long t0 = clock64(); !done && clock64() - t0 < limit;) done = bar_test(at, 0u);
  if (!done) *reinterpret_cast<volatile int *>(dead) = 1;
  __syncwarp();
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

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
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

__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// Which of the 32 keys from `at` on token n sees (sees() for all of them).
__device__ __forceinline__ uint32_t seen_word(const AttnParams &p, const KeyRange &k, int b, int n,
                                              int at) {
  const uint32_t in_ctx = low_bits(k.ctx - at);
  uint32_t w = in_ctx, block = ~in_ctx;
  const int place = p.window ? k.ctx + clamp_pos(p, b, n) : 0;
  // the window's first place; no difference of two places leaves 32 bits
  if (p.window) w &= low_bits(p.sinks - at) | ~low_bits(max(place - p.window + 1, at) - at);
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

// What a masked tile of values needs before its product: tokens that were not
// copied (not in `valid`) become zero, and so do infinities and NaNs, which
// nonfinite_values adds to the rows that see them.  Thread t of `threads`; tokens
// from `from` on.
template <class E, int D>
__device__ __forceinline__ void clean_values(char *entry, uint4 valid, int from, int t, int threads,
                                             int *bad) {
  using W = Entry<D>;
  constexpr int kPer = W::kGroup / 16;  // pieces of eight tokens
  constexpr uint32_t exps = E::kExp * 0x10001u, ones = (E::kExp & (0u - E::kExp)) * 0x10001u;
  auto key_of = [](int i) { return i / kPer * 8 + i / 8 % 8; };
  auto piece = [&](int i) { return reinterpret_cast<uint4 *>(entry + i * 16); };
  const int count = __popc(valid.x) + __popc(valid.y) + __popc(valid.z) + __popc(valid.w);
  const bool prefix = valid.x == low_bits(count) && valid.y == low_bits(count - 32) &&
                      valid.z == low_bits(count - 64) && valid.w == low_bits(count - 96);
  int i = from / 8 * kPer + t;
  // tokens that were copied, four pieces at once; an exponent of all ones
  // carries into the sign's place
  const int copied = prefix ? count / 8 * kPer : 0;
  for (; i + 3 * threads < copied; i += 4 * threads) {
    uint32_t found = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 y = *piece(i + j * threads);
      found |= ((y.x & exps) + ones) | ((y.y & exps) + ones) | ((y.z & exps) + ones) |
               ((y.w & exps) + ones);
    }
    if (!(found & 0x80008000u)) continue;
    for (int j = 0; j < 4; ++j) {
      uint4 *x = piece(i + j * threads);
      *x = make_uint4(finite_or_zero<E>(x->x), finite_or_zero<E>(x->y), finite_or_zero<E>(x->z),
                      finite_or_zero<E>(x->w));
    }
    *reinterpret_cast<volatile int *>(bad) = 1;
  }
  for (; i < W::kBytes / 16; i += threads) {
    const int key = key_of(i);
    const uint32_t word = key < 64 ? (key < 32 ? valid.x : valid.y) : (key < 96 ? valid.z : valid.w);
    uint4 *x = piece(i);
    if (!((word >> (key & 31)) & 1u)) {
      *x = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint4 y = *x;
    if ((((y.x & exps) + ones) | ((y.y & exps) + ones) | ((y.z & exps) + ones) |
         ((y.w & exps) + ones)) &
        0x80008000u) {
      *x = make_uint4(finite_or_zero<E>(y.x), finite_or_zero<E>(y.y), finite_or_zero<E>(y.z),
                      finite_or_zero<E>(y.w));
      *reinterpret_cast<volatile int *>(bad) = 1;
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// The first token of a masked tile that clean_values has to look at: those
// before it are copied and every row sees them.
__device__ __forceinline__ int clean_from(const AttnParams &p, const KeyRange &k, int at0,
                                          uint4 valid) {
  if (p.window) return 0;
  const int from = min(max(k.all - at0, 0), kTileKeys);
  const uint32_t missing = (low_bits(from) & ~valid.x) | (low_bits(from - 32) & ~valid.y) |
                           (low_bits(from - 64) & ~valid.z) | (low_bits(from - 96) & ~valid.w);
  return missing ? 0 : from;
}

__device__ __forceinline__ bool tile_masked(const AttnParams &p, const UnitWalk &u, int at0,
                                            uint4 valid) {
  return (valid.x & valid.y & valid.z & valid.w) != 0xFFFFFFFFu ||
         !all_seen(p, u.k, at0, kTileKeys);
}
__device__ __forceinline__ uint4 both(uint4 a, uint4 b) {
  return make_uint4(a.x & b.x, a.y & b.y, a.z & b.z, a.w & b.w);
}
// Which of the tile's keys token n sees, as far as that is known before its
// pages are.
__device__ __forceinline__ uint4 seen_tile(const AttnParams &p, const UnitWalk &u, int n, int at0) {
  if (all_seen(p, u.k, at0, kTileKeys))
    return make_uint4(0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu);
  return make_uint4(seen_word(p, u.k, u.b, n, at0), seen_word(p, u.k, u.b, n, at0 + 32),
                    seen_word(p, u.k, u.b, n, at0 + 64), seen_word(p, u.k, u.b, n, at0 + 96));
}

// One row per thread: the scores of a tile become weights, m and l go on, the
// row's outputs so far are rescaled where m is raised (`first`: there are none).
// seen: the keys that the row sees; masked: some are missing in some row.
template <class E, int D>
__device__ __forceinline__ void softmax_tile(float c, bool mine, bool masked, uint4 seen,
                                             uint32_t s_at, uint32_t o_at, bool first, float &m,
                                             float &l) {
  tc_after();
  uint32_t s[4][32];
  float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  const uint32_t vis[4] = {seen.x, seen.y, seen.z, seen.w};
  tm_load32(s[0], s_at);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    tm_wait_ld();
    if (j < 3) tm_load32(s[j + 1], s_at + (j + 1) * 32);
    if (masked) {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (!(vis[j] & (1u << e))) s[j][e] = __float_as_uint(-INFINITY);
    }
#pragma unroll
    for (int e = 0; e < 32; e += 2)
      x[j] = max3(x[j], __uint_as_float(s[j][e]), __uint_as_float(s[j][e + 1]));
  }
  float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * c;
  if constexpr (E::kNarrow) top -= kLift;
  const bool raise = mine && top > m + kSlack;
  if (__any_sync(0xFFFFFFFFu, raise)) {
    const float to = raise ? top : m;
    const float f = m == -INFINITY ? 0.f : fast_exp2(m - to);
    l *= f;
    m = to;
    if (!first) {
      // the products before S's are complete: O is whole
#pragma unroll 1
      for (int d = 0; d < D; d += 16) {
        uint32_t o[16];
        tm_load16(o, o_at + d);
        tm_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tm_store16(o_at + d, o);
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
      float2 y =
          fma2(make_float2(__uint_as_float(s[j][e]), __uint_as_float(s[j][e + 1])), c2, sub2);
      y.x = fast_exp2(y.x);
      y.y = fast_exp2(y.y);
      sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], y);
      // the product takes the weights in the cache's type: each is off by at
      // most half a step of that type, as the values themselves are (float16: or
      // by 2^-32 of the row's largest, which the sum of weights does not see)
      packed[e / 2] = E::pack(y.x, y.y);
    }
    tm_store16(s_at + j * 16, packed);
  }
  sum[0] = add2(sum[0], sum[1]);
  l += sum[0].x + sum[0].y;
  tm_wait_st();
}

// The same for a quarter of the tile's keys, those of the warp's part: weights of
// zero for the other quarters' keys.  seen: of the 32 keys.
template <class E, int D>
__device__ __forceinline__ void softmax_part(float c, bool mine, bool masked, uint32_t seen,
                                             int part, uint32_t s_at, uint32_t o_at, bool first,
                                             float &m, float &l) {
  tc_after();
  uint32_t s[32];
  tm_load32(s, s_at + part * 32);
  tm_wait_ld();
  if (masked) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!(seen & (1u << e))) s[e] = __float_as_uint(-INFINITY);
  }
  float x[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < 32; e += 2)
    x[(e >> 1) & 1] = max3(x[(e >> 1) & 1], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
  float top = fmaxf(x[0], x[1]) * c;
  if constexpr (E::kNarrow) top -= kLift;
  const bool raise = mine && top > m + kSlack;
  if (__any_sync(0xFFFFFFFFu, raise)) {
    const float to = raise ? top : m;
    const float f = m == -INFINITY ? 0.f : fast_exp2(m - to);
    l *= f;
    m = to;
    if (!first) {
#pragma unroll 1
      for (int d = 0; d < D; d += 16) {
        uint32_t o[16];
        tm_load16(o, o_at + d);
        tm_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tm_store16(o_at + d, o);
      }
    }
  }
  const float sub = m == -INFINITY ? 0.f : -m;
  const float2 c2 = make_float2(c, c), sub2 = make_float2(sub, sub);
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  uint32_t packed[16], none[16];
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float2 y = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, sub2);
    y.x = fast_exp2(y.x);
    y.y = fast_exp2(y.y);
    sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], y);
    packed[e / 2] = E::pack(y.x, y.y);
    none[e / 2] = 0u;
  }
#pragma unroll
  for (int j = 1; j < 4; ++j) tm_store16(s_at + ((part + j) & 3) * 16, none);
  tm_store16(s_at + part * 16, packed);
  sum[0] = add2(sum[0], sum[1]);
  l += sum[0].x + sum[0].y;
  tm_wait_st();
}

// 32 bytes of a row at once: a whole sector.
__device__ __forceinline__ void store32(void *p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// A row's end: its outputs from tensor memory, divided by the sum, or its piece
// of a cut unit.  By whole warps; `mine`: the row exists.
template <class E, int D>
__device__ __forceinline__ void write_row(const AttnParams &p, const UnitWalk &u, int worker, int row,
                                          int n, bool mine, uint32_t o_at, float m, float l,
                                          bool bad) {
  using TE = typename E::T;
  const bool whole = u.whole();
  float *slot = p.part + piece_slot(u, worker) * slot_floats(p.rows, D);
  float *slot_o = slot + slot_stats(p.rows) + static_cast<size_t>(row) * D;
  const bool wide_out = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
  const long long at = mine ? out_row(p, u.b, u.h, u.r0 + row) : 0;
  TE *out = static_cast<TE *>(p.out) + at * D;
  const float norm = l == 0.f ? 0.f : (whole ? 1.f / l : 1.f);
  tc_after();
#pragma unroll 1
  for (int d = 0; d < D; d += 32) {
    __syncwarp();
    uint32_t o[32];
    tm_load32(o, o_at + d);
    tm_wait_ld();
    if (mine) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        o[i] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(o[i]) * norm);
      if (whole) {
#pragma unroll
        for (int e = 0; e < 32; e += 16) {
          uint32_t v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[i] = E::pack(__uint_as_float(o[e + 2 * i]), __uint_as_float(o[e + 2 * i + 1]));
          if (wide_out) {
            store32(out + d + e, v);
          } else {
            *reinterpret_cast<uint4 *>(out + d + e) = make_uint4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<uint4 *>(out + d + e + 8) = make_uint4(v[4], v[5], v[6], v[7]);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          const uint32_t v[8] = {o[e],     o[e + 1], o[e + 2], o[e + 3],
                                 o[e + 4], o[e + 5], o[e + 6], o[e + 7]};
          store32(slot_o + d + e, v);
        }
      }
    }
  }
  if (bad && mine && l != 0.f) {
    for (int d = 0; d < D; d += 4) {
      const float4 v =
          nonfinite_values<TE, kTileKeys>(p, u, n, d, make_float4(0.f, 0.f, 0.f, 0.f));
      const float x[4] = {v.x, v.y, v.z, v.w};
      for (int e = 0; e < 4; ++e) {
        if (x[e] == 0.f) continue;
        if (whole) {
          out[d + e] = E::from(E::to(out[d + e]) + x[e]);
        } else {
          slot_o[d + e] += x[e];
        }
      }
    }
  }
  if (mine) {
    if (!whole) {
      slot[row] = m;
      slot[p.rows + row] = l;
    } else if (p.lse) {
      p.lse[at] = row_lse(m, l);
    }
  }
  __syncwarp();
  tc_before();
}

// Where the quarters of a split unit's rows meet.
struct Quarters {
  static constexpr int kFloats = 1024;  // of a warp
  float o[4][kFloats];
  float ml[4][2][32];
};

// The end of a unit whose rows are spread over four quarters; by the stream's
// four warps.  Few rows meet at once (8 of 128 outputs, 16 of 64), more rows 32
// outputs at a time, a row's 16-byte pieces permuted so that eight rows meet
// eight banks.  False: a wait gave up.
template <class E, int D>
__device__ __forceinline__ bool write_split(const AttnParams &p, const UnitWalk &u, int worker,
                                            int part, int lane, uint32_t o_at, float m, float l,
                                            Quarters &x, const void *meet, uint32_t &met, int *dead,
                                            const int *bad) {
  using TE = typename E::T;
  constexpr int kFew = Quarters::kFloats / D;
  const bool whole = u.whole();
  const int live = u.live_rows(p), t = part * 32 + lane;
  const bool few = live <= kFew;
  // this thread's eight outputs of a pass
  const int row = few ? t / (D / 8) : t / 4, d0 = few ? t % (D / 8) * 8 : t % 4 * 8;
  const int pitch = few ? D : 32, mask = few ? 0 : row & 7;
  float *slot = p.part + piece_slot(u, worker) * slot_floats(p.rows, D);
  x.ml[part][0][lane] = m;
  x.ml[part][1][lane] = l;
  tc_after();
  float M = -INFINITY, sum = 0.f, f[4];
  for (int pass = 0; pass < (few ? 1 : D / 32); ++pass) {
#pragma unroll 1
    for (int d = few ? 0 : pass * 32; d < (few ? D : pass * 32 + 32); d += 32) {
      __syncwarp();
      uint32_t o[32];
      tm_load32(o, o_at + d);
      tm_wait_ld();
      if (lane < live) {
        float *to = x.o[part] + lane * pitch + (few ? d : 0);
        const int swap = few ? 0 : lane & 7;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<uint4 *>(to + (e ^ swap) * 4) =
              make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      }
    }
    __syncwarp();
    if (lane == 0) bar_arrive(meet);
    if (!warp_wait(meet, met++ & 1u, dead)) return false;
    if (row < live) {
      if (pass == 0) {
#pragma unroll
        for (int w = 0; w < 4; ++w) M = fmaxf(M, x.ml[w][0][row]);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          // an empty quarter has l zero; one of NaN scores has m -infinity too
          const float lw = x.ml[w][1][row];
          f[w] = lw == 0.f ? 0.f : fast_exp2(x.ml[w][0][row] - M);
          sum += f[w] * lw;
        }
      }
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 y = *reinterpret_cast<const float4 *>(x.o[w] + row * pitch +
                                                             (((d0 >> 2) + e) ^ mask) * 4);
          v[4 * e] += f[w] * y.x;
          v[4 * e + 1] += f[w] * y.y;
          v[4 * e + 2] += f[w] * y.z;
          v[4 * e + 3] += f[w] * y.w;
        }
      }
      const int d = pass * 32 + d0;
      if (*reinterpret_cast<const volatile int *>(bad)) {
#pragma unroll 1
        for (int e = 0; e < 8; e += 4) {
          const float4 y = nonfinite_values<TE, kTileKeys>(p, u, (u.r0 + row) / p.G, d + e,
                                                           make_float4(0.f, 0.f, 0.f, 0.f));
          if (e == 0) {
            v[0] += y.x, v[1] += y.y, v[2] += y.z, v[3] += y.w;
          } else {
            v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
          }
        }
      }
      if (whole) {
        const long long at = out_row(p, u.b, u.h, u.r0 + row);
        const float n = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = sum == 0.f ? 0.f : v[e] * n;
        *reinterpret_cast<uint4 *>(static_cast<TE *>(p.out) + at * D + d) = make_uint4(
            E::pack(v[0], v[1]), E::pack(v[2], v[3]), E::pack(v[4], v[5]), E::pack(v[6], v[7]));
        if (d == 0 && p.lse) p.lse[at] = row_lse(M, sum);
      } else {
        float *to = slot + slot_stats(p.rows) + static_cast<size_t>(row) * D + d;
        store4(to, make_float4(v[0], v[1], v[2], v[3]));
        store4(to + 4, make_float4(v[4], v[5], v[6], v[7]));
        if (d == 0) {
          slot[row] = M;
          slot[p.rows + row] = sum;
        }
      }
    }
    // the quarters are read before they are written again
    __syncwarp();
    if (lane == 0) bar_arrive(meet);
    if (!warp_wait(meet, met++ & 1u, dead)) return false;
  }
  tc_before();
  return true;
}

// Tokens of a box: the largest power of two, up to a tile, that divides the page
// size.  A tile begins at a multiple of it, so a box never leaves its page.  (32 trees
// of 60 nodes on pages of 24 tokens, 16 boxes of 8 a tile: 115 us, 110 on pages of 64
// and 1031 in rows16_kernel; one token within windows there 58 us, 54 in
// rows16_kernel, on pages of 16 45.)
__host__ __device__ __forceinline__ int box_tokens(int page_size) {
  const int two = page_size & -page_size;
  return two < kTileKeys ? two : kTileKeys;
}

// The boxes of a tile of keys or values, one per lane.
struct BoxLoader {
  const CUtensorMap *map;
  int unit_page, unit_head, unit_token;
  int box, boxes, shift;  // tokens of a box, boxes of a tile, log2(tokens)

  __device__ __forceinline__ BoxLoader(const AttnParams &p, const WideMaps &maps, bool values) {
    map = values ? &maps.v : &maps.k;
    unit_page = values ? maps.v_page : maps.k_page;
    unit_head = values ? maps.v_head : maps.k_head;
    unit_token = values ? maps.v_token : maps.k_token;
    box = box_tokens(p.C.page_size);
    boxes = kTileKeys / box;
    shift = 31 - __clz(box);
  }
  // This lane's page of tile i of the unit, -1 where it has none.
  __device__ __forceinline__ int page(const AttnParams &p, const UnitWalk &u, int i, int lane) const {
    const int at = key_tile(u.k, u.i0 + i) * kTileKeys + lane * box;
    if (lane >= boxes || i >= u.i1 - u.i0 || at >= u.k.end) return -1;
    // between the sinks and the window
    if (at >= p.sinks && at + box <= u.k.first) return -1;
    return page_at(p.S, u.b, p.C.page_size == box ? at >> shift : at / p.C.page_size);
  }
  // Which of the 32 tokens from 32 * j of the tile at at0 on are copied.
  __device__ __forceinline__ uint32_t valid_word(const UnitWalk &u, uint32_t pages, int at0,
                                                 int j) const {
    if (pages == low_bits(boxes) && at0 + kTileKeys <= u.k.end) return 0xFFFFFFFFu;
    uint32_t word = 0u;
    for (int k = 0; k < 32; k += box)
      if ((pages >> ((j * 32 + k) >> shift)) & 1u) word |= low_bits(box) << k;
    return word & low_bits(u.k.end - at0 - j * 32);
  }
  // By a whole warp, into an entry that is free.
  template <int D>
  __device__ __forceinline__ void load(const AttnParams &p, const UnitWalk &u, int at0, int page_id,
                                       uint32_t pages, uint32_t entry, const void *full,
                                       int lane) const {
    using W = Entry<D>;
    __syncwarp();
    if (lane == 0) bar_expect(full, __popc(pages) * box * W::kRow * W::kPanels);
    __syncwarp();
    if ((pages >> lane) & 1u) {
      const int token = p.C.page_size == box ? 0 : (at0 + lane * box) % p.C.page_size;
      box_load(entry + lane * (box >> 3) * W::kGroup, map, full, 0, 0, 0, 0,
               page_id * unit_page + u.h * unit_head + token * unit_token);
    }
  }
};

// S = Q K^T of a tile, by a whole warp; qpanel: bytes of a panel of queries.
template <class E, int D>
__device__ __forceinline__ void issue_scores(uint32_t s, uint32_t q_at, int qpanel, uint32_t k_at) {
  using W = Entry<D>;
  constexpr uint32_t idesc = mma_idesc<E>(kTileKeys, false);
  // a descriptor's address counts 16 bytes
  const uint64_t a = smem_desc(q_at, 16, 1024), b = smem_desc(k_at, 16, W::kGroup);
  tc_after();
  if (elect_one()) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      mma_ss(s, a + ((k >> 2) * qpanel + (k & 3) * 32) / 16,
             b + ((k >> 2) * W::kPanel + (k & 3) * 32) / 16, idesc, k > 0);
  }
  __syncwarp();
}
// O (+)= P V.
template <class E, int D>
__device__ __forceinline__ void issue_outputs(uint32_t o, uint32_t p_at, uint32_t v_at, bool first) {
  using W = Entry<D>;
  constexpr uint32_t idesc = mma_idesc<E>(D, true);
  const uint64_t b = smem_desc(v_at, W::kPanel, W::kGroup);
  tc_after();
  if (elect_one()) {
#pragma unroll
    for (int k = 0; k < kTileKeys / 16; ++k)
      mma_ts(o, p_at + k * 8, b + k * 2 * W::kGroup / 16, idesc, !first || k > 0);
  }
  __syncwarp();
}
__device__ __forceinline__ void issue_commit(const void *bar) {
  if (elect_one()) mma_commit(bar);
  __syncwarp();
}

// By the warp that frees it; other warps see the address behind a barrier.
__device__ __forceinline__ void tm_alloc(void *slot) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                   smem_u32(slot))
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  tc_before();
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tm_free(uint32_t tmem, int warp) {
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 11)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// A wait gave up: the copies into a ring of entries, and of the queries, land before
// the CTA ends.  The loaders may have made them all without a wait that failed, so
// this is for when every role has left its loops; by a whole warp.  sent[x]: entries
// of the numbers x, x + 2, ... below it were asked for.  Entries leave the ring in
// order, so those before the last kRing have landed.
struct Sent {
  uint32_t entries[2], queries;
};
template <int kRing>
__device__ __forceinline__ void land_copies(const unsigned long long (&full)[kRing],
                                            const unsigned long long *q_full, const Sent &sent) {
  const uint32_t top = max(sent.entries[0], sent.entries[1]);
  for (uint32_t i = 0; i < kRing && i < top; ++i) {
    const uint32_t e = top - 1 - i;
    if (e < sent.entries[e & 1]) bar_linger(&full[e % kRing], (e / kRing) & 1u);
  }
  if (sent.queries > 0) bar_linger(q_full, (sent.queries - 1) & 1u);
}

// A wait gave up: the rows of the run's units become NaN, whatever was written of
// them, or the sums of their pieces of cut units, which the join then carries to
// the rows; and their sequences are flagged.  By the whole CTA.
template <class E, int D>
__device__ __noinline__ void void_run(const AttnParams &p, const Line &line) {
  using TE = typename E::T;
  const float nan = __int_as_float(0x7FC00000);
  UnitWalk v;
  if (!v.start(p, line)) return;
  do {
    const int live = v.live_rows(p);
    float *slot = p.part + piece_slot(v, line.worker) * slot_floats(p.rows, D);
    for (int i = threadIdx.x; i < live * (D / 4); i += kWideThreads) {
      const int row = i / (D / 4), d = i % (D / 4) * 4;
      const long long at = out_row(p, v.b, v.h, v.r0 + row);
      if (v.whole()) store4(static_cast<TE *>(p.out) + at * D + d, make_float4(nan, nan, nan, nan));
      if (d > 0) continue;
      if (!v.whole()) {
        slot[row] = -INFINITY;
        slot[p.rows + row] = nan;
      } else if (p.lse) {
        p.lse[at] = nan;
      }
    }
    if (threadIdx.x == 0 && p.flags) atomicOr(p.flags + v.b, SPEC_FLAG_TIMEOUT);
  } while (v.next(p, line));
}

// ---------------------------------------------------------------------------
// two streams with units of their own
// ---------------------------------------------------------------------------

// kSplit: at most 32 rows, spread over the four quarters.
template <int D, bool kSplit>
struct SoloCtl {
  // entries of a stream: what 227 KB hold beside the queries and the quarters
  static constexpr int kRing = D == 128 ? 2 : (kSplit ? 5 : 6);
  struct Stream {
    unsigned long long full[kRing], empty[kRing], s_full, p_full, o_done, q_full, q_empty, meet,
        drain;
    alignas(16) uint32_t valid[kValidRing][4];
    Sent sent;
  } stream[2];
  RunScratch<kWideThreads, 2> runs;
  uint32_t tmem;
  int dead, bad;
};
template <int D, bool kSplit>
struct SoloShape {
  static constexpr int kQPanel = 128 * 128, kQ = Entry<D>::kPanels * kQPanel;  // of a stream
  static constexpr int kRing = SoloCtl<D, kSplit>::kRing;
  static constexpr int kEntries = 2 * kQ;  // where the rings begin
  static constexpr int kMeet = kEntries + 2 * kRing * Entry<D>::kBytes;
  static constexpr int kCtl = kMeet + (kSplit ? 2 * static_cast<int>(sizeof(Quarters)) : 0);
  static constexpr int kSmem = kCtl + static_cast<int>(sizeof(SoloCtl<D, kSplit>));
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

}  // namespace

template <class E, int D, bool kSplit>
__global__ void __launch_bounds__(kWideThreads, 1)
    solo_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ WideMaps maps) {
  using W = Entry<D>;
  using Shape = SoloShape<D, kSplit>;
  using Ctl = SoloCtl<D, kSplit>;
  constexpr int kRing = Shape::kRing;
  // all shared memory is this array, so its alignment is the swizzle's
  extern __shared__ __align__(1024) char wide_s[];
  Ctl &ctl = *reinterpret_cast<Ctl *>(wide_s + Shape::kCtl);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);

  if (tid < 2) {
    auto &st = ctl.stream[tid];
    for (int i = 0; i < kRing; ++i) {
      bar_init(&st.full[i], 1);
      bar_init(&st.empty[i], 1);
    }
    bar_init(&st.s_full, 1);
    bar_init(&st.p_full, 4);
    bar_init(&st.o_done, 1);
    bar_init(&st.q_full, 1);
    bar_init(&st.q_empty, 1);
    bar_init(&st.meet, 4);
    bar_init(&st.drain, 1);
    ctl.dead = 0;
    ctl.bad = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 11) tm_alloc(&ctl.tmem);
  if (warp == 8 && lane == 0) {
    prefetch_map(&maps.k);
    prefetch_map(&maps.v);
    prefetch_map(&maps.q);
  }
  __syncwarp();
  Line lines[2];
  // barriers as well; consecutive workers on different CTAs
  find_runs(p, ctl.runs, blockIdx.x, gridDim.x, lines);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // of this warp's stream
  const int g = warp < 8 ? warp >> 2 : warp & 1;
  const Line line = g ? lines[1] : lines[0];
  UnitWalk u;
  const bool busy = u.start(p, line);
  if (lane == 0 && (warp == 8 || warp == 9)) write_join(p, line, busy ? &u : nullptr);
  tc_after();
  const uint32_t tmem = ctl.tmem;
  if (lines[0].w0 == lines[0].w1 && lines[1].w0 == lines[1].w1) {
    tm_free(tmem, warp);
    return;
  }
  auto &st = ctl.stream[g];
  const uint32_t s_at = tmem + g * 128, o_at = tmem + 256 + g * 128;
  const uint32_t q_at = smem_u32(wide_s) + g * Shape::kQ;
  char *ring = wide_s + Shape::kEntries + g * kRing * W::kBytes;
  const uint32_t ring_at = smem_u32(ring);
  bool ok = true;

  if (warp < 8) {
    // -------------------------------------------------------------- softmax
    more_regs<kSoftRegs>();
    const int part = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(part * 32) << 16;
    // a split stream's lane holds the same row in every warp
    const int row = kSplit ? lane : tid & 127;
    Quarters &quarters = reinterpret_cast<Quarters *>(wide_s + Shape::kMeet)[kSplit ? g : 0];
    uint32_t tiles = 0, units = 0, met = 0;
    if (busy) do {
        const int n_tiles = u.i1 - u.i0, live = u.live_rows(p);
        const bool mine = row < live, works = kSplit || part * 32 < live;
        const int n = (u.r0 + min(row, live - 1)) / p.G;
        const int idle = kSplit ? 0 : 4 - min((live + 31) / 32, 4);  // warps without rows
        float m = -INFINITY, l = 0.f;
        for (int i = 0; i < n_tiles; ++i, ++tiles) {
          const int at0 = key_tile(u.k, u.i0 + i) * kTileKeys;
          uint4 seen = make_uint4(0, 0, 0, 0);
          if (kSplit) {
            seen.x = all_seen(p, u.k, at0, kTileKeys)
                         ? 0xFFFFFFFFu
                         : seen_word(p, u.k, u.b, n, at0 + part * 32);
          } else if (works) {
            seen = seen_tile(p, u, n, at0);
          }
          if (!(ok = warp_wait(&st.s_full, tiles & 1u, &ctl.dead))) break;
          const uint4 valid = *reinterpret_cast<const uint4 *>(st.valid[tiles % kValidRing]);
          const bool masked = tile_masked(p, u, at0, valid);
          if (kSplit) {
            const uint32_t word = part < 2 ? (part == 0 ? valid.x : valid.y)
                                           : (part == 2 ? valid.z : valid.w);
            softmax_part<E, D>(p.scale_log2, mine, masked, seen.x & word, part, s_at + lanes,
                               o_at + lanes, i == 0, m, l);
          } else if (works) {
            softmax_tile<E, D>(p.scale_log2, mine, masked, both(seen, valid), s_at + lanes,
                               o_at + lanes, i == 0, m, l);
          }
          if (masked && (idle == 0 || !works)) {
            const uint32_t e = 2 * tiles + 1;
            if (!(ok = warp_wait(&st.full[e % kRing], (e / kRing) & 1u, &ctl.dead))) break;
            clean_values<E, D>(ring + e % kRing * W::kBytes, valid, clean_from(p, u.k, at0, valid),
                               idle == 0 ? tid & 127 : (part - (4 - idle)) * 32 + lane,
                               idle == 0 ? 128 : idle * 32, &ctl.bad);
          }
          tc_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&st.p_full);
        }
        if (!ok || !(ok = warp_wait(&st.o_done, units++ & 1u, &ctl.dead))) break;
        if constexpr (kSplit) {
          if (!(ok = write_split<E, D>(p, u, line.worker, part, lane, o_at + lanes, m, l, quarters,
                                       &st.meet, met, &ctl.dead, &ctl.bad)))
            break;
        } else if (works) {
          write_row<E, D>(p, u, line.worker, row, n, mine, o_at + lanes, m, l,
                          *reinterpret_cast<volatile int *>(&ctl.bad) != 0);
        }
      } while (u.next(p, line));
  } else {
    fewer_regs<kRestRegs>();
    if (warp < 10) {
    // ------------------------------------------------ queries, keys, values
    const BoxLoader keys(p, maps, false), values(p, maps, true);
    uint32_t tiles = 0, units = 0, sent = 0;
    if (busy) do {
        const int n_tiles = u.i1 - u.i0;
        int page = keys.page(p, u, 0, lane), next = keys.page(p, u, 1, lane);
        for (int i = 0; ok && i < n_tiles; ++i, ++tiles) {
          // a tile's pages are looked up two tiles ahead
          const int behind = keys.page(p, u, i + 2, lane);
          const uint32_t pages = __ballot_sync(0xFFFFFFFFu, page_ok(p.C, page));
          const int at0 = key_tile(u.k, u.i0 + i) * kTileKeys;
          uint32_t e = 2 * tiles;
          if (!(ok = warp_wait(&st.empty[e % kRing], ((e / kRing) & 1u) ^ 1u, &ctl.dead))) break;
          if (lane < 4) st.valid[tiles % kValidRing][lane] = keys.valid_word(u, pages, at0, lane);
          keys.load<D>(p, u, at0, page, pages, ring_at + e % kRing * W::kBytes, &st.full[e % kRing],
                       lane);
          sent = e + 1;
          if (i == 0) {
            // once the products of the unit before have read theirs
            if (!(ok = warp_wait(&st.q_empty, (units & 1u) ^ 1u, &ctl.dead))) break;
            ++units;
            if (lane == 0) {
              constexpr int kRows = kSplit ? 32 : 128, kCopies = 128 / kRows;
              bar_expect(&st.q_full, kCopies * (kRows / p.G * p.G) * W::kRow * W::kPanels);
              for (int x = 0; x < W::kPanels * kCopies; ++x)
                box_load(q_at + x / kCopies * Shape::kQPanel + x % kCopies * kRows * W::kRow, &maps.q,
                         &st.q_full, 0, 0, u.r0 / p.G, x / kCopies,
                         u.b * maps.q_seq + u.h * maps.q_head);
            }
          }
          ++e;
          if (!(ok = warp_wait(&st.empty[e % kRing], ((e / kRing) & 1u) ^ 1u, &ctl.dead))) break;
          values.load<D>(p, u, at0, page, pages, ring_at + e % kRing * W::kBytes,
                         &st.full[e % kRing], lane);
          sent = e + 1;
          page = next;
          next = behind;
        }
      } while (ok && u.next(p, line));
    if (lane == 0) st.sent = Sent{{sent, sent}, units};
    } else {
    // ------------------------------------------------------------- products
    uint32_t tiles = 0, units = 0;
    if (busy) first_wait(&st.full[0], p.first_wait, &ctl.dead);
    if (busy) do {
        const int n_tiles = u.i1 - u.i0;
        for (int i = 0; i < n_tiles; ++i, ++tiles) {
          uint32_t e = 2 * tiles;
          if (!(ok = warp_wait(&st.full[e % kRing], (e / kRing) & 1u, &ctl.dead))) break;
          if (i == 0 && !(ok = warp_wait(&st.q_full, units++ & 1u, &ctl.dead))) break;
          issue_scores<E, D>(s_at, q_at, Shape::kQPanel, ring_at + e % kRing * W::kBytes);
          issue_commit(&st.s_full);
          issue_commit(&st.empty[e % kRing]);
          if (i + 1 == n_tiles) issue_commit(&st.q_empty);
          ++e;
          if (!(ok = warp_wait(&st.full[e % kRing], (e / kRing) & 1u, &ctl.dead))) break;
          if (!(ok = warp_wait(&st.p_full, tiles & 1u, &ctl.dead))) break;
          issue_outputs<E, D>(o_at, s_at, ring_at + e % kRing * W::kBytes, i == 0);
          if (i + 1 == n_tiles) issue_commit(&st.o_done);
          issue_commit(&st.empty[e % kRing]);
        }
      } while (ok && u.next(p, line));
    // nothing is in flight when the tensor memory goes back
    issue_commit(&st.drain);
    bar_linger(&st.drain, 0u);
    }
  }
  tm_free(tmem, warp);
  if (!ctl.dead) return;
  if (warp == 8 || warp == 9) land_copies(st.full, &st.q_full, st.sent);
  void_run<E, D>(p, lines[0]);
  void_run<E, D>(p, lines[1]);
}

namespace {

// ---------------------------------------------------------------------------
// two streams that share keys and values
// ---------------------------------------------------------------------------

template <int D>
struct PairCtl {
  static constexpr int kRing = D == 128 ? 5 : 12;  // what 227 KB hold beside the queries
  // checked: an entry of values is ready for its products
  unsigned long long full[kRing], empty[kRing], checked[kRing], s_full[2], p_full[2], o_done[2],
      q_full, q_empty, drain;
  alignas(16) uint32_t valid[kValidRing][4];
  RunScratch<kWideThreads, 1> runs;
  Sent sent;
  uint32_t tmem;
  int dead, bad;
};
template <int D>
struct PairShape {
  static constexpr int kQPanel = 128 * 128, kQ = Entry<D>::kPanels * kQPanel;  // of a row tile
  static constexpr int kRing = PairCtl<D>::kRing;
  static constexpr int kEntries = 2 * kQ;
  static constexpr int kCtl = kEntries + kRing * Entry<D>::kBytes;
  static constexpr int kSmem = kCtl + static_cast<int>(sizeof(PairCtl<D>));
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

}  // namespace

template <class E, int D>
__global__ void __launch_bounds__(kWideThreads, 1)
    pair_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ WideMaps maps) {
  using W = Entry<D>;
  using Shape = PairShape<D>;
  using Ctl = PairCtl<D>;
  constexpr int kRing = Shape::kRing;
  extern __shared__ __align__(1024) char wide_s[];
  char *ring = wide_s + Shape::kEntries;
  Ctl &ctl = *reinterpret_cast<Ctl *>(wide_s + Shape::kCtl);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int tile_rows = p.rows / 2;

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      bar_init(&ctl.full[i], 1);
      bar_init(&ctl.empty[i], 2);  // the products and the check are done with it
      bar_init(&ctl.checked[i], 1);
    }
    for (int g = 0; g < 2; ++g) {
      bar_init(&ctl.s_full[g], 1);
      bar_init(&ctl.p_full[g], 4);
      bar_init(&ctl.o_done[g], 1);
    }
    bar_init(&ctl.q_full, 1);
    bar_init(&ctl.q_empty, 1);
    bar_init(&ctl.drain, 1);
    ctl.dead = 0;
    ctl.bad = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 11) tm_alloc(&ctl.tmem);
  if (warp == 8 && lane == 0) {
    prefetch_map(&maps.k);
    prefetch_map(&maps.v);
    prefetch_map(&maps.q);
  }
  __syncwarp();
  Line lines[1];
  find_runs(p, ctl.runs, blockIdx.x, 0, lines);  // barriers as well
  const Line &line = lines[0];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  UnitWalk u;
  const bool busy = u.start(p, line);
  if (tid == 0) write_join(p, line, busy ? &u : nullptr);
  tc_after();
  const uint32_t tmem = ctl.tmem;
  if (!busy) {  // the same for every thread
    tm_free(tmem, warp);
    return;
  }
  const uint32_t ring_at = smem_u32(ring), q_at = smem_u32(wide_s);
  uint32_t tiles = 0, units = 0;
  bool ok = true;

  if (warp < 8) {
    // -------------------------------------------------------------- softmax
    more_regs<kSoftRegs>();
    const int g = warp >> 2, part = warp & 3, tile_row = tid & 127, row = g * tile_rows + tile_row;
    const uint32_t lanes = static_cast<uint32_t>(part * 32) << 16;
    const uint32_t s_at = tmem + lanes + g * 128, o_at = tmem + lanes + 256 + g * 128;
    uint32_t turns = 0, ended = 0;  // tiles and units of this stream
    do {
      const int n_tiles = u.i1 - u.i0, live = u.live_rows(p);
      const int rows = min(tile_rows, live - g * tile_rows);  // of this stream
      const bool mine = tile_row < rows, works = part * 32 < rows;
      const int n = (u.r0 + min(row, live - 1)) / p.G;
      float m = -INFINITY, l = 0.f;
      for (int i = 0; rows > 0 && i < n_tiles; ++i) {
        const int at0 = key_tile(u.k, u.i0 + i) * kTileKeys;
        uint4 seen = make_uint4(0, 0, 0, 0);
        if (works) seen = seen_tile(p, u, n, at0);
        if (!(ok = warp_wait(&ctl.s_full[g], turns++ & 1u, &ctl.dead))) break;
        if (works) {
          const uint4 valid = *reinterpret_cast<const uint4 *>(ctl.valid[(tiles + i) % kValidRing]);
          softmax_tile<E, D>(p.scale_log2, mine, tile_masked(p, u, at0, valid), both(seen, valid),
                             s_at, o_at, i == 0, m, l);
        }
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&ctl.p_full[g]);
      }
      if (!ok) break;
      tiles += n_tiles;
      if (rows > 0) {
        if (!(ok = warp_wait(&ctl.o_done[g], ended++ & 1u, &ctl.dead))) break;
        if (works)
          write_row<E, D>(p, u, line.worker, row, n, mine, o_at, m, l,
                          *reinterpret_cast<volatile int *>(&ctl.bad) != 0);
      }
    } while (u.next(p, line));
  } else {
    fewer_regs<kRestRegs>();
    if (warp < 10) {
    // ------------------------------ warp 8: keys and queries, warp 9: values
    const bool values = warp == 9;
    const BoxLoader boxes(p, maps, values);
    uint32_t sent = 0;
    do {
      const int n_tiles = u.i1 - u.i0, live = u.live_rows(p);
      // a tile's pages are looked up two tiles ahead
      int page = boxes.page(p, u, 0, lane), next = boxes.page(p, u, 1, lane);
      for (int i = 0; ok && i < n_tiles; ++i, ++tiles) {
        const int behind = boxes.page(p, u, i + 2, lane);
        const uint32_t pages = __ballot_sync(0xFFFFFFFFu, page_ok(p.C, page));
        const int at0 = key_tile(u.k, u.i0 + i) * kTileKeys;
        const uint32_t e = 2 * tiles + (values ? 1 : 0);
        if (!(ok = warp_wait(&ctl.empty[e % kRing], ((e / kRing) & 1u) ^ 1u, &ctl.dead))) break;
        if (!values && lane < 4)
          ctl.valid[tiles % kValidRing][lane] = boxes.valid_word(u, pages, at0, lane);
        boxes.load<D>(p, u, at0, page, pages, ring_at + e % kRing * W::kBytes, &ctl.full[e % kRing],
                      lane);
        sent = e + 1;
        if (!values && i == 0) {
          // once the products of the unit before have read theirs
          if (!(ok = warp_wait(&ctl.q_empty, (units & 1u) ^ 1u, &ctl.dead))) break;
          ++units;
          if (lane == 0) {
            const int used = live > tile_rows ? 2 : 1;
            bar_expect(&ctl.q_full, used * tile_rows * W::kRow * W::kPanels);
            for (int t = 0; t < used; ++t)
              for (int x = 0; x < W::kPanels; ++x)
                box_load(q_at + t * Shape::kQ + x * Shape::kQPanel, &maps.q, &ctl.q_full, 0, 0,
                         (u.r0 + t * tile_rows) / p.G, x, u.b * maps.q_seq + u.h * maps.q_head);
          }
        }
        page = next;
        next = behind;
      }
    } while (ok && u.next(p, line));
    if (lane == 0) {
      ctl.sent.entries[values] = sent;
      if (!values) ctl.sent.queries = units;
    }
    } else if (warp == 10) {
    // -------------------------------------------------- values made ready
    first_wait(&ctl.full[0], p.first_wait, &ctl.dead);
    do {
      const int n_tiles = u.i1 - u.i0;
      for (int i = 0; i < n_tiles; ++i, ++tiles) {
        uint32_t e = 2 * tiles;
        if (!(ok = warp_wait(&ctl.full[e % kRing], (e / kRing) & 1u, &ctl.dead))) break;
        const int at0 = key_tile(u.k, u.i0 + i) * kTileKeys;
        const uint4 valid = *reinterpret_cast<const uint4 *>(ctl.valid[tiles % kValidRing]);
        if (lane == 0) {
          bar_arrive(&ctl.checked[e % kRing]);  // every entry is a phase of its place
          bar_arrive(&ctl.empty[e % kRing]);
        }
        ++e;
        // only an entry that has landed is this warp's to release
        if (!(ok = warp_wait(&ctl.full[e % kRing], (e / kRing) & 1u, &ctl.dead))) break;
        if (tile_masked(p, u, at0, valid)) {
          clean_values<E, D>(ring + e % kRing * W::kBytes, valid,
                             clean_from(p, u.k, at0, valid), lane, 32, &ctl.bad);
        }
        __syncwarp();
        if (lane == 0) {
          bar_arrive(&ctl.checked[e % kRing]);
          bar_arrive(&ctl.empty[e % kRing]);
        }
      }
    } while (ok && u.next(p, line));
    } else {
    // ------------------------------------------------------------- products
    uint32_t made[2] = {0, 0};  // tiles of each stream
    auto take = [&](uint32_t e) {  // an entry that has landed
      ok = warp_wait(&ctl.full[e % kRing], (e / kRing) & 1u, &ctl.dead);
      return ring_at + e % kRing * W::kBytes;
    };
    auto scores = [&](int g, uint32_t k_at) {
      issue_scores<E, D>(tmem + g * 128, q_at + g * Shape::kQ, Shape::kQPanel, k_at);
      issue_commit(&ctl.s_full[g]);
    };
    do {
      const int n_tiles = u.i1 - u.i0, streams = u.live_rows(p) > tile_rows ? 2 : 1;
      uint32_t k_at = take(2 * tiles);
      if (!ok || !(ok = warp_wait(&ctl.q_full, units++ & 1u, &ctl.dead))) break;
      for (int g = 0; g < streams; ++g) scores(g, k_at);
      issue_commit(&ctl.empty[2 * tiles % kRing]);
      if (n_tiles == 1) issue_commit(&ctl.q_empty);
      for (int i = 0; ok && i < n_tiles; ++i, ++tiles) {
        const uint32_t e = 2 * tiles + 1;
        const bool more = i + 1 < n_tiles;
        const uint32_t v_at = take(e);
        if (!ok || !(ok = warp_wait(&ctl.checked[e % kRing], (e / kRing) & 1u, &ctl.dead))) break;
        for (int g = 0; ok && g < streams; ++g) {
          if (!(ok = warp_wait(&ctl.p_full[g], made[g]++ & 1u, &ctl.dead))) break;
          issue_outputs<E, D>(tmem + 256 + g * 128, tmem + g * 128, v_at, i == 0);
          if (!more) issue_commit(&ctl.o_done[g]);
          if (g == streams - 1) issue_commit(&ctl.empty[e % kRing]);
          if (more) {
            if (g == 0) k_at = take(e + 1);
            if (!ok) break;
            scores(g, k_at);
            if (g == streams - 1) {
              issue_commit(&ctl.empty[(e + 1) % kRing]);
              if (i + 2 == n_tiles) issue_commit(&ctl.q_empty);
            }
          }
        }
      }
    } while (ok && u.next(p, line));
    // nothing is in flight when the tensor memory goes back
    issue_commit(&ctl.drain);
    bar_linger(&ctl.drain, 0u);
    }
  }
  tm_free(tmem, warp);
  if (!ctl.dead) return;
  if (warp == 8) land_copies(ctl.full, &ctl.q_full, ctl.sent);
  void_run<E, D>(p, line);
}

namespace {

bool wide_pairs(const AttnParams &p) { return p.rows > wide_tile_rows(p.G); }
int wide_ctas(const AttnParams &p) { return wide_pairs(p) ? p.workers : p.workers / 2; }
// As many rows as a quarter of the lanes holds.  Split and not: one token at
// B = 256 325 and 343 us, in windows of 1024 at B = 64 44 and 74, eight tokens at
// B = 64 (32 rows) 107 and 112.
bool solo_splits(const AttnParams &p) { return p.S.N * p.G <= 32; }

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
// tokens, origin]; a box is box_tokens() of a page.
bool cache_map(CUtensorMap *map, Origin *o, int dtype, const KvCache &C, int D, const char *base,
               long long page, long long token, long long head) {
  const long long strides[3] = {page, head, token};
  const int tokens = box_tokens(C.page_size);
  const long long sizes[3] = {C.pages, C.heads, C.page_size > tokens ? C.page_size : 1};
  if (!origin(o, strides, sizes)) return false;
  const cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(D / 64),
                              static_cast<cuuint64_t>(tokens / 8),
                              static_cast<cuuint64_t>(o->count)};
  const long long steps[4] = {token, 128, 8 * token, o->step};
  const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(D / 64),
                             static_cast<cuuint32_t>(tokens / 8), 1};
  return encode_map(map, dtype, base, dims, steps, box);
}

template <auto kKernel>
cudaError_t start_wide(int smem, const AttnParams &p, const WideMaps &maps, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  return launch_large(kKernel, done, smem, wide_ctas(p), kWideThreads, smem, stream, p, maps);
}

template <class E, int D>
cudaError_t start_wide(const AttnParams &p, const WideMaps &maps, cudaStream_t stream) {
  if (wide_pairs(p)) return start_wide<pair_kernel<E, D>>(PairShape<D>::kSmem, p, maps, stream);
  if (solo_splits(p))
    return start_wide<solo_kernel<E, D, true>>(SoloShape<D, true>::kSmem, p, maps, stream);
  return start_wide<solo_kernel<E, D, false>>(SoloShape<D, false>::kSmem, p, maps, stream);
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
  const int rows = !wide_pairs(p) && solo_splits(p) ? 32 : 128;
  const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(rows / p.G),
                             1, 1};
  return encode_map(&maps->q, dtype, p.q, dims, steps, box);
}

cudaError_t launch_attention_wide(const AttnParams &p, const WideMaps &maps, int dtype,
                                  cudaStream_t stream) {
  if (dtype == SPEC_BF16)
    return p.D == 64 ? start_wide<Bf16, 64>(p, maps, stream) : start_wide<Bf16, 128>(p, maps, stream);
  return p.D == 64 ? start_wide<F16, 64>(p, maps, stream) : start_wide<F16, 128>(p, maps, stream);
}

}  // namespace sv
