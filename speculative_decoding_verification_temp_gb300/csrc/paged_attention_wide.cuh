// What the attention kernels with asynchronous copies, mbarriers and tensor memory
// share: bounded waits, the fifth-generation matrix instructions, the softmax of a row
// per thread and the ends of units.
#pragma once

#include "paged_attention.cuh"
#include "q4.cuh"

namespace sv {

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
// What the operands made of a 4-bit cache are multiplied by; scores and outputs take the
// factor back.  Values of 2^-10 and more keep all of float16's bits.
constexpr float kFourth = 1.f / 16.f;

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
// shortened it; by the warp that has just asked for them.  The others find in their own
// waits, or at the run's end, that it gave up.  limit <= 0: a test at the moment of
// asking, which finds nothing; it is not made, since an instruction fetch in between
// can take as long as the keys do.
__device__ __forceinline__ void first_wait(const void *bar, long long limit, int *dead) {
  if (limit >= kWaitCycles) return;
  const uint32_t at = smem_u32(bar);
  bool done = false;
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
// seen: the keys that the row sees; masked: some are missing in some row; outputs_whole:
// called by whole warps before the outputs so far are scaled, false where a wait gave up.
template <class E, int D, class F>
__device__ __forceinline__ void softmax_tile(float c, bool mine, bool masked, uint4 seen,
                                             uint32_t s_at, uint32_t o_at, bool first, float &m,
                                             float &l, const F &outputs_whole) {
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
    if (!first && outputs_whole()) {
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
template <class E, int D, class F>
__device__ __forceinline__ void softmax_part(float c, bool mine, bool masked, uint32_t seen,
                                             int part, uint32_t s_at, uint32_t o_at, bool first,
                                             float &m, float &l, const F &outputs_whole) {
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
    if (!first && outputs_whole()) {
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

__device__ __forceinline__ uint32_t word_at(const char *p) { return *reinterpret_cast<const uint32_t *>(p); }

// Two outputs of token n that the keys' values which are not finite add, from the parts
// of tiles that some row does not see whole; see nonfinite_values.
template <int D, int kSlice>
static __device__ __noinline__ float2 nonfinite_values_q4(const AttnParams &p, const UnitWalk u, int n,
                                                          int d) {
  float a[2] = {0.f, 0.f};
  for (int i = u.i0; i < u.i1; ++i) {
    const int t0 = key_tile(u.k, i) << p.tile_log2;
    for (int at0 = t0; at0 < t0 + (1 << p.tile_log2) && at0 < u.k.end; at0 += kSlice) {
      bool whole = all_seen(p, u.k, at0, kSlice);
      for (int at = at0; at < at0 + kSlice && whole; ++at)
        whole = at < u.k.end && page_ok(p.C, page_at(p.S, u.b, at / p.C.page_size));
      if (whole) continue;
      for (int at = at0; at < min(at0 + kSlice, u.k.end); ++at) {
        const int index = at / p.C.page_size, page = page_at(p.S, u.b, index);
        if (!page_ok(p.C, page) || !sees(p, u.k, u.b, n, at)) continue;
        const char *row = p.C.v + page * p.C.v_page + (at - index * p.C.page_size) * p.C.v_token +
                          u.h * p.C.v_head;
        const uint32_t pair = word_at(row + D / 2 + d / (D / 4) * 4);
        if (q4_finite(pair)) continue;
        const float2 s = q4_pair(pair);
        float x[8];
        q4_codes(word_at(row + d / 8 * 4), x);
        for (int j = 0; j < 2; ++j) a[j] += fmaf(s.x, x[d % 8 + j], s.y);
      }
    }
  }
  return make_float2(a[0], a[1]);
}

// What values that are not finite add to outputs d to d + 3 of token n's rows.
template <class E, int D, bool kFour>
__device__ __forceinline__ float4 nonfinite_row(const AttnParams &p, const UnitWalk &u, int n, int d) {
  if constexpr (kFour) {
    const float2 a = nonfinite_values_q4<D, 32>(p, u, n, d);
    const float2 b = nonfinite_values_q4<D, 32>(p, u, n, d + 2);
    return make_float4(a.x, a.y, b.x, b.y);
  } else {
    return nonfinite_values<typename E::T, kTileKeys>(p, u, n, d, make_float4(0.f, 0.f, 0.f, 0.f));
  }
}

// A row's end: its outputs from tensor memory, divided by the sum, or its piece
// of a cut unit.  By whole warps; `mine`: the row exists; kFour: of a 4-bit cache.
template <class E, int D, bool kFour = false>
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
  const float norm = l == 0.f ? 0.f : (whole ? 1.f / l : 1.f) * (kFour ? 1.f / kFourth : 1.f);
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
      const float4 v = nonfinite_row<E, D, kFour>(p, u, n, d);
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
template <class E, int D, bool kFour = false>
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
          if constexpr (kFour) f[w] *= 1.f / kFourth;
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
          const float4 y = nonfinite_row<E, D, kFour>(p, u, (u.r0 + row) / p.G, d + e);
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
template <int kWarp = 11>
__device__ __forceinline__ void tm_free(uint32_t tmem, int warp) {
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == kWarp)
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
template <class E, int D, int kCta = kWideThreads>
__device__ __noinline__ void void_run(const AttnParams &p, const Line &line) {
  using TE = typename E::T;
  const float nan = __int_as_float(0x7FC00000);
  UnitWalk v;
  if (!v.start(p, line)) return;
  do {
    const int live = v.live_rows(p);
    float *slot = p.part + piece_slot(v, line.worker) * slot_floats(p.rows, D);
    for (int i = threadIdx.x; i < live * (D / 4); i += kCta) {
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

}  // namespace sv
