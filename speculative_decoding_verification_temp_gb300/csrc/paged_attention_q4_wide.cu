// Attention over a paged cache of 4-bit rows (q4.cuh) for more than 8 rows of queries, on
// the fifth-generation tensor cores: units of one row tile, at most 128 rows (new tokens
// times the group's heads; at most 32 are held by each of the four quarters of the lanes),
// or pairs of tiles, as solo_kernel and pair_kernel of the 16-bit caches.
//
// Six warps make the products' operands: each copies 32 keys and then their values for
// itself, reads the codes into registers and writes the values m + s n as float16 into the
// entries of a ring (half a step of 2^-11, against quantisation by half a step of 1/15 of a
// group's spread).  The softmax threads bring the queries, as float16 scaled by a power of
// two where a row's largest leaves 2^14.  One warp issues the products, two warpgroups turn
// scores into weights, a thread a row.  Every hand-over is an mbarrier, every wait is
// bounded.
//
// Bound by the turns of making, scores, softmax and outputs, not by a unit of the SM
// (issue slots 0.33, tensor pipe 0.23 active).  A tile of 128 keys of one unit of eight
// tokens (32/8 heads of 128, B = 64, 1..4096 tokens: 118 us) takes about 3200 cycles, without
// its making 2700; of a pair (60-node trees, B = 32: 119 us) 4900, without it 4700.
#include "q4_copies.cuh"

namespace sv {

namespace {

// For more than 32 rows: two warpgroups of softmax, six warps that make operands, one that
// issues products; the last of the fourth warpgroup has nothing to do.
constexpr int kThreads4 = 512, kMakers = 6, kIssuer = 8 + kMakers;
// Registers of a softmax thread and of the others: 256 * 184 + 256 * 72 are the 512 * 128
// that the CTA is launched with.
constexpr int kSoftRegs4 = 184, kRestRegs4 = 72;

// For at most 32 rows: two warpgroups of softmax, six warps that make operands, one that
// issues products.
constexpr int kSplitMakers = 6, kSplitIssuer = 8 + kSplitMakers, kSplitThreads = 32 * (kSplitIssuer + 1);

// Hand-overs of a ring of entries.
template <int kSize>
struct Ring4 {
  static constexpr int kRing = kSize;
  unsigned long long full[kRing], empty[kRing];
  alignas(16) uint32_t valid[kValidRing][4];
  __device__ __forceinline__ void init() {
    for (int i = 0; i < kRing; ++i) {
      bar_init(&full[i], kTileKeys / kQ4Keys);
      bar_init(&empty[i], 1);
    }
  }
};
// Hand-overs of a stream.
struct Stream4 {
  unsigned long long s_full, p_full, o_done;
  __device__ __forceinline__ void init() {
    bar_init(&s_full, 1);
    bar_init(&p_full, 4);
    bar_init(&o_done, 1);
  }
};
// Rows as they are, copied by a maker for itself.
template <int D>
struct Raw4 {
  static constexpr int kWarp = Q4Copies<q4_row_bytes(D)>::kBytes;
};

template <int D>
struct PairCtl4 {
  Ring4<D == 128 ? 4 : 8> ring;
  Stream4 stream[2];
  unsigned long long q_full, q_empty, drain;
  RunScratch<kThreads4, 1> runs;
  uint32_t tmem;
  int dead, bad;
};
template <int D, int kThreads>
struct SoloCtl4 {
  Ring4<D == 128 ? 4 : 8> ring;
  // of a group's even and odd tiles, in turn: outputs of a tile that is not the last one
  // are waited for only where they are scaled, and its phase is not mistaken for the one
  // before
  struct {
    unsigned long long s_full[2], p_full[2], o_done[2], q_full, q_empty, meet;
  } group[2];
  unsigned long long drain;
  RunScratch<kThreads, 1> runs;
  uint32_t tmem;
  int dead, bad;
};
template <int D>
struct Shape4 {
  static constexpr int kQPanel = 128 * 128, kQ = Entry<D>::kPanels * kQPanel;  // of a row tile
  static constexpr int kEntries = 2 * kQ;
  static constexpr int kRing = D == 128 ? 4 : 8;  // entries, of both streams together
  static constexpr int kRaw = kEntries + kRing * Entry<D>::kBytes;
  static constexpr int kCtl = kRaw + kMakers * Raw4<D>::kWarp;
  static constexpr int kPair = kCtl + static_cast<int>(sizeof(PairCtl4<D>));
  static constexpr int kSplitEntries = kQ, kSplitRaw = kSplitEntries + kRing * Entry<D>::kBytes;
  static constexpr int kMeet = kSplitRaw + kSplitMakers * Raw4<D>::kWarp;
  static constexpr int kSplitCtl = kMeet + 2 * static_cast<int>(sizeof(Quarters));
  static constexpr int kSplit = kSplitCtl + static_cast<int>(sizeof(SoloCtl4<D, kThreads4>));
  static_assert(kPair <= 227 * 1024 && kSplit <= 227 * 1024, "shared memory of a CTA");
};

__device__ __forceinline__ __half2 half2_of(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t word_of(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }

// The operands are values times kFourth (paged_attention_wide.cuh), 2^-4.  A nibble at
// bits 6 to 9 is a float16 below its normal ones, n 2^-18, exactly: with a scale of s 2^14,
// for s below 4 (a group that spans less than 60), a value takes a shift, a mask and half
// of a fused multiply and add.  (Any form that takes larger scales too has twice the
// instructions of float16, which run at a quarter of the rate.)
__device__ __forceinline__ uint4 word_values(uint32_t w, __half2 scale, __half2 low) {
  auto value = [&](uint32_t x) { return word_of(__hfma2(half2_of(x & 0x03C003C0u), scale, low)); };
  return make_uint4(value(w << 6), value(w << 2), value(w >> 2), value(w >> 6));
}
// A scale of 4 and more is taken as it is, with n 2^-4 instead.
__device__ __forceinline__ bool large_scale(uint32_t pair) { return (pair & 0x7FFFu) >= 0x4400u; }
// Large scales and others, in groups of one row or in rows of one warp.
__device__ __forceinline__ uint4 word_values_any(uint32_t w, uint32_t pair) {
  const bool large = large_scale(pair);
  const __half2 up = __float2half2_rn(large ? 16384.f : 1.f);
  const __half2 f = __hmul2(half2_of(pair), __floats2half2_rn(large ? 1.f : kFourth * 262144.f, kFourth));
  const __half2 scale = __low2half2(f), low = __high2half2(f);
  auto value = [&](uint32_t x) { return word_of(__hfma2(__hmul2(half2_of(x & 0x03C003C0u), up), scale, low)); };
  return make_uint4(value(w << 6), value(w << 2), value(w >> 2), value(w >> 6));
}

// A row of queries as float16 into its place of a tile (panels of 64 values, the
// 128-byte swizzle), by one thread; returns the factor that the row's scores take.  Rows
// whose largest lies within 2^-4 .. 2^14 stay as they are, others are brought there by a
// power of two: float16's step below its normal values, 2^-24, is then 2^-20 of the largest.
// By whole warps: `mine`: there is such a row; ready: the place may be written, false where
// a wait gave up.
template <class E, int D, class F>
__device__ __forceinline__ float put_query(const char *from, bool mine, float scale, char *tile, int panel_bytes,
                                           int row, const F &ready) {
  using TE = typename E::T;
  uint4 v[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) v[i] = mine ? *reinterpret_cast<const uint4 *>(from + i * 16) : make_uint4(0, 0, 0, 0);
  float top = 0.f;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = fabsf(E::to(reinterpret_cast<const TE *>(&v[i])[e]));
      odd |= !(x < INFINITY);
      top = fmaxf(top, x);
    }
  const int exponent = top > 16384.f || (top > 1e-30f && top < 0.0625f) ? min(max(8 - ilogbf(top), -126), 126) : 0;
  // a query that is not finite makes its row's scores NaN, those that the mask leaves
  const float up = __int_as_float((127 + exponent) << 23);
  if (!ready()) return 0.f;
#pragma unroll
  for (int i = 0; mine && i < D / 8; ++i) {
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const TE *x = reinterpret_cast<const TE *>(&v[i]) + 2 * e;
      h[e] = odd ? 0x7E007E00u : F16::pack(E::to(x[0]) * up, E::to(x[1]) * up);
    }
    *reinterpret_cast<uint4 *>(tile + i / 8 * panel_bytes + row * 128 + (((i & 7) ^ (row & 7)) << 4)) =
        make_uint4(h[0], h[1], h[2], h[3]);
  }
  return scale * (1.f / kFourth) * (odd ? 1.f : __int_as_float((127 - exponent) << 23));
}

// The rows of a stream, a thread each: their queries, their weights and their outputs.
// first_row: of the stream in a unit; by the stream's four warps.
template <class E, int D, int kRing>
__device__ __forceinline__ void weigh_rows(const AttnParams &p, const Line &line, UnitWalk u, int part, int lane,
                                           int first_row, int tile_rows, uint32_t s_at, uint32_t o_at,
                                           char *q_tile, Stream4 &st, const void *q_full, const void *q_empty,
                                           Ring4<kRing> &ring, int *dead, int *bad) {
  const int tile_row = part * 32 + lane, row = first_row + tile_row;
  s_at += static_cast<uint32_t>(part * 32) << 16;
  o_at += static_cast<uint32_t>(part * 32) << 16;
  uint32_t tiles = 0, units = 0;
  bool ok = true;
  uint32_t turns = 0, ended = 0;  // tiles and units of this stream
  float c = 0.f;
  // This thread's row of the next unit's queries, once the products of the unit before
  // have read theirs.  Its outputs are written behind that, while the next unit's first
  // products run.
  auto bring_queries = [&](const UnitWalk &w) {
    const bool has = row < w.live_rows(p) && tile_row < tile_rows;
    const int r = w.r0 + (has ? row : 0), n = r / p.G;
    c = put_query<E, D>(p.q + w.b * p.q_seq + n * p.q_token + (w.h * p.G + r - n * p.G) * p.q_head, has,
                        p.scale_log2, q_tile, Shape4<D>::kQPanel, tile_row,
                        [&] { return ok = warp_wait(q_empty, (units & 1u) ^ 1u, dead); });
    if (!ok) return;
    ++units;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) bar_arrive(q_full);
  };
  bring_queries(u);
  for (bool more = true; ok && more;) {
    const int n_tiles = u.i1 - u.i0, live = u.live_rows(p);
    const int rows = min(tile_rows, live - first_row);  // of this stream
    const bool mine = tile_row < rows, works = part * 32 < rows;
    const int n = (u.r0 + min(row, live - 1)) / p.G;
    float m = -INFINITY, l = 0.f;
    for (int i = 0; rows > 0 && i < n_tiles; ++i) {
      const int at0 = key_tile(u.k, u.i0 + i) * kTileKeys;
      uint4 seen = make_uint4(0, 0, 0, 0);
      if (works) seen = seen_tile(p, u, n, at0);
      if (!(ok = warp_wait(&st.s_full, turns++ & 1u, dead))) break;
      if (works) {
        const uint4 valid = *reinterpret_cast<const uint4 *>(ring.valid[(tiles + i) % kValidRing]);
        softmax_tile<F16, D>(c, mine, tile_masked(p, u, at0, valid), both(seen, valid), s_at, o_at,
                             i == 0, m, l, [] { return true; });
      }
      tc_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&st.p_full);
    }
    if (!ok) break;
    tiles += n_tiles;
    const UnitWalk v = u;
    more = u.next(p, line);
    if (more) bring_queries(u);
    if (rows > 0) {
      if (!ok || !(ok = warp_wait(&st.o_done, ended++ & 1u, dead))) break;
      if (works)
        write_row<E, D, true>(p, v, line.worker, row, n, mine, o_at, m, l,
                              *reinterpret_cast<volatile int *>(bad) != 0);
    }
  }
}

// A stream's or a pair's operands, by kCount warps of which this is the maker-th: they
// take 32 keys and their values in turn, keys into an entry, then values into the next.
// The warp copies keys behind those that it has made while it makes the values, and the
// other way round.
template <int D, int kCount, int kRing>
__device__ __forceinline__ void make_operands(const AttnParams &p, const Line &line, UnitWalk u, int maker,
                                              int lane, char *raw, char *entries, Ring4<kRing> &ring,
                                              int *dead, int *bad) {
  using W = Entry<D>;
  constexpr int kRow = q4_row_bytes(D);
  uint32_t tiles = 0;
  bool ok = true;
  constexpr int kParts = kTileKeys / kQ4Keys;
  using Copies = Q4Copies<kRow, kCount * kQ4Keys>;
  Copies copies(p, lane);
  const uint32_t raw_at = smem_u32(raw);
  // a pass makes 32 16-byte pieces of codes, of eight neighbouring rows each (which
  // meet eight banks, in the rows as in the swizzle)
  constexpr int kPieces = D / 32, kPasses = kPieces, kOwn = 32 / kPieces;
  const int own = D == 128 ? lane & 7 : (lane & 7) + (lane >> 4) * 8;
  const int piece = D == 128 ? lane >> 3 : (lane >> 3) & 1;
  uint32_t done = 0;  // parts before the unit, of all makers
  do {
    const int n_tiles = u.i1 - u.i0, parts = n_tiles * kParts;
    auto at_of = [&](int part) {
      return key_tile(u.k, u.i0 + part / kParts) * kTileKeys + part % kParts * kQ4Keys;
    };
    // this warp's parts: first, first + kCount, ...
    const int first = (maker + kCount - static_cast<int>(done % kCount)) % kCount;
    copies.begin(p, u, at_of(first), lane);
    uint32_t word = 0u;  // of the next part
    // (the first turn makes none)
#pragma unroll 1
    for (int part = first - kCount; ok && part < parts; part += kCount) {
      const uint32_t tile = tiles + part / kParts, there = word;
      const int quarter = part % kParts, at0 = at_of(part), ahead = part + kCount;
      const bool masked = there != 0xFFFFFFFFu || !all_seen(p, u.k, at0, kQ4Keys);
      const char *rows = raw;
#pragma unroll 1
      for (int values = 0; values < 2; ++values, rows += kQ4Keys * kRow) {
       if (part >= 0) {
        copy_wait<1>();
        const uint32_t e = 2 * tile + values;
        if (!(ok = warp_wait(&ring.empty[e % kRing], ((e / kRing) & 1u) ^ 1u, dead))) break;
        __syncwarp();
        if (!values && lane == 0) ring.valid[tile % kValidRing][quarter] = there;
        // 32 values are half of a panel's row
        char *entry = entries + e % kRing * W::kBytes + quarter * (kQ4Keys / 8) * W::kGroup + piece / 2 * W::kPanel;
#pragma unroll 1
        for (int x = 0; x < kPasses; ++x) {
          const int key = x * kOwn + own, r = key & 7;
          const char *row = rows + key * kRow;
          const uint4 codes = *reinterpret_cast<const uint4 *>(row + piece * 16);
          uint32_t pair[2];
          if constexpr (D == 128) {
            pair[0] = word_at(row + D / 2 + piece * 4);
            pair[1] = pair[0];
          } else {
            pair[0] = word_at(row + D / 2 + piece * 8);
            pair[1] = word_at(row + D / 2 + piece * 8 + 4);
          }
          if (masked) {
            // rows that were not copied stand for zeros, and so do groups that are not
            // finite, which nonfinite_values_q4 adds
            const bool copied = (there >> key) & 1u;
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (!copied || (values && !q4_finite(pair[j]))) {
                if (copied) *reinterpret_cast<volatile int *>(bad) = 1;
                pair[j] = 0u;
              }
          }
          char *to = entry + key / 8 * W::kGroup + r * W::kRow;
          const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
          auto put = [&](int j, uint4 v) {
            *reinterpret_cast<uint4 *>(to + ((((piece & 1) * 4 + j) ^ r) << 4)) = v;
          };
          if (__any_sync(0xFFFFFFFFu, large_scale(pair[0]) || large_scale(pair[1]))) {
#pragma unroll 1
            for (int j = 0; j < 4; ++j)
              put(j, word_values_any(word_at(row + piece * 16 + j * 4), j < 2 ? pair[0] : pair[1]));
          } else {
            uint32_t f[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
              f[j] = word_of(__hmul2(half2_of(pair[j]), __floats2half2_rn(kFourth * 262144.f, kFourth)));
#pragma unroll
            for (int j = 0; j < 4; ++j)
              put(j, word_values(w[j], half2_of(__byte_perm(f[j >> 1], 0, 0x1010)),
                                 half2_of(__byte_perm(f[j >> 1], 0, 0x3232))));
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive(&ring.full[e % kRing]);
       }
        // the rows are read: those ahead may take their place, while the others are made
        if (ahead < parts) word = copies.template ask<false>(p, u, at_of(ahead), raw_at, lane, values);
        copy_commit();
      }
      if (!ok) break;
      if (done == 0 && part == 0) first_wait(&ring.full[0], p.first_wait, dead);
    }
    tiles += n_tiles;
    done += parts;
  } while (ok && u.next(p, line));
  copy_wait<0>();
}

}  // namespace

template <class E, int D>
__global__ void __launch_bounds__(kThreads4, 1) pair4_kernel(const __grid_constant__ AttnParams p) {
  using W = Entry<D>;
  using Shape = Shape4<D>;
  using Ctl = PairCtl4<D>;
  constexpr int kRing = Shape::kRing;
  extern __shared__ __align__(1024) char wide4_s[];
  char *ring = wide4_s + Shape::kEntries;
  Ctl &ctl = *reinterpret_cast<Ctl *>(wide4_s + Shape::kCtl);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int tile_rows = p.rows / 2;

  if (tid == 0) {
    ctl.ring.init();
    ctl.stream[0].init();
    ctl.stream[1].init();
    bar_init(&ctl.q_full, 8);
    bar_init(&ctl.q_empty, 1);
    bar_init(&ctl.drain, 1);
    ctl.dead = 0;
    ctl.bad = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssuer) tm_alloc(&ctl.tmem);
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
    tm_free<kIssuer>(tmem, warp);
    return;
  }
  const uint32_t ring_at = smem_u32(ring), q_at = smem_u32(wide4_s);
  uint32_t tiles = 0, units = 0;
  bool ok = true;

  if (warp < 8) {
    // -------------------------------------------------------------- softmax
    more_regs<kSoftRegs4>();
    const int g = warp >> 2;
    weigh_rows<E, D>(p, line, u, warp & 3, lane, g * tile_rows, tile_rows, tmem + g * 128, tmem + 256 + g * 128,
                     wide4_s + g * Shape::kQ, ctl.stream[g], &ctl.q_full, &ctl.q_empty, ctl.ring, &ctl.dead,
                     &ctl.bad);
  } else {
    fewer_regs<kRestRegs4>();
    if (warp < 8 + kMakers) {
      // ------------------------------------------------- operands of the products
      make_operands<D, kMakers>(p, line, u, warp - 8, lane, wide4_s + Shape::kRaw + (warp - 8) * Raw4<D>::kWarp,
                                ring, ctl.ring, &ctl.dead, &ctl.bad);
    } else if (warp == kIssuer) {
      // ------------------------------------------------------------- products
      uint32_t made[2] = {0, 0};  // tiles of each stream
      auto take = [&](uint32_t e) {  // an entry that is ready
        ok = warp_wait(&ctl.ring.full[e % kRing], (e / kRing) & 1u, &ctl.dead);
        return ring_at + e % kRing * W::kBytes;
      };
      auto scores = [&](int g, uint32_t k_at) {
        issue_scores<F16, D>(tmem + g * 128, q_at + g * Shape::kQ, Shape::kQPanel, k_at);
        issue_commit(&ctl.stream[g].s_full);
      };
      do {
        const int n_tiles = u.i1 - u.i0, streams = u.live_rows(p) > tile_rows ? 2 : 1;
        uint32_t k_at = take(2 * tiles);
        if (!ok || !(ok = warp_wait(&ctl.q_full, units++ & 1u, &ctl.dead))) break;
        for (int g = 0; g < streams; ++g) scores(g, k_at);
        issue_commit(&ctl.ring.empty[2 * tiles % kRing]);
        if (n_tiles == 1) issue_commit(&ctl.q_empty);
        for (int i = 0; ok && i < n_tiles; ++i, ++tiles) {
          const uint32_t e = 2 * tiles + 1;
          const bool more = i + 1 < n_tiles;
          const uint32_t v_at = take(e);
          if (!ok) break;
          for (int g = 0; ok && g < streams; ++g) {
            if (!(ok = warp_wait(&ctl.stream[g].p_full, made[g]++ & 1u, &ctl.dead))) break;
            issue_outputs<F16, D>(tmem + 256 + g * 128, tmem + g * 128, v_at, i == 0);
            if (!more) issue_commit(&ctl.stream[g].o_done);
            if (g == streams - 1) issue_commit(&ctl.ring.empty[e % kRing]);
            if (more) {
              if (g == 0) k_at = take(e + 1);
              if (!ok) break;
              scores(g, k_at);
              if (g == streams - 1) {
                issue_commit(&ctl.ring.empty[(e + 1) % kRing]);
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
  tm_free<kIssuer>(tmem, warp);
  if (!ctl.dead) return;
  void_run<E, D, kThreads4>(p, line);
}

// Units of one row tile.  kSplit: of at most 32 rows: each quarter of the lanes holds them
// all and weighs a quarter of a tile's keys, and the quarters are added at the unit's end.
// Otherwise a thread has a row (sixteen tokens of 32/8 heads at B = 64 148 us, as one
// stream of pair4_kernel 167).  Scores have two places: a tile's products with the keys run
// while the tile before is in its softmax.  Two warpgroups take the units in turn: one
// writes a unit while the other has the next.
template <class E, int D, bool kSplit>
__global__ void __launch_bounds__(kSplit ? kSplitThreads : kThreads4, 1)
    solo4_kernel(const __grid_constant__ AttnParams p) {
  using W = Entry<D>;
  using Shape = Shape4<D>;
  constexpr int kRing = Shape::kRing, kThreads = kSplit ? kSplitThreads : kThreads4;
  using Ctl = SoloCtl4<D, kThreads>;
  extern __shared__ __align__(1024) char wide4_s[];
  Ctl &ctl = *reinterpret_cast<Ctl *>(wide4_s + Shape::kSplitCtl);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  if (tid == 0) {
    ctl.ring.init();
    for (auto &x : ctl.group) {
      for (int i = 0; i < 2; ++i) {
        bar_init(&x.s_full[i], 1);
        bar_init(&x.p_full[i], 4);
        bar_init(&x.o_done[i], 1);
      }
      bar_init(&x.q_full, 4);
      bar_init(&x.q_empty, 1);
      bar_init(&x.meet, 4);
    }
    bar_init(&ctl.drain, 1);
    ctl.dead = 0;
    ctl.bad = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kSplitIssuer) tm_alloc(&ctl.tmem);
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
    tm_free<kSplitIssuer>(tmem, warp);
    return;
  }
  char *entries = wide4_s + Shape::kSplitEntries;
  bool ok = true;

  if (warp < 8) {
    // -------------------------------------------------------------- softmax
    if constexpr (!kSplit) more_regs<kSoftRegs4>();
    const int g = warp >> 2, part = warp & 3, row = kSplit ? lane : part * 32 + lane;
    auto &x = ctl.group[g];
    const uint32_t lanes = tmem + (static_cast<uint32_t>(part * 32) << 16), o_at = lanes + 256 + g * 128;
    Quarters &quarters = reinterpret_cast<Quarters *>(wide4_s + Shape::kMeet)[g];
    uint32_t t = 0, own = 0, units = 0, met = 0;  // tiles, of this group, units of this group
    int unit = 0;
    auto outputs_done = [&](uint32_t of) { return ok = warp_wait(&x.o_done[of & 1], (of >> 1) & 1u, &ctl.dead); };
    do {
      const int n_tiles = u.i1 - u.i0, live = u.live_rows(p);
      if ((unit++ & 1) != g) {
        t += n_tiles;
        continue;
      }
      const bool mine = row < live, works = kSplit || part * 32 < live;
      const int r = u.r0 + min(row, live - 1), n = r / p.G;
      // once the products of the unit before, the other group's, have read theirs
      const float c = put_query<E, D>(
          p.q + u.b * p.q_seq + n * p.q_token + (u.h * p.G + r - n * p.G) * p.q_head, mine, p.scale_log2, wide4_s,
          Shape::kQPanel, part * 32 + lane, [&] {
            if (unit > 1) ok = warp_wait(&ctl.group[g ^ 1].q_empty, (units + g - 1) & 1u, &ctl.dead);
            return ok;
          });
      if (!ok) break;
      ++units;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive(&x.q_full);
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < n_tiles; ++i, ++t, ++own) {
        const int at0 = key_tile(u.k, u.i0 + i) * kTileKeys;
        uint4 seen = make_uint4(0, 0, 0, 0);
        if (kSplit) {
          seen.x = all_seen(p, u.k, at0, kTileKeys) ? 0xFFFFFFFFu : seen_word(p, u.k, u.b, n, at0 + part * 32);
        } else if (works) {
          seen = seen_tile(p, u, n, at0);
        }
        if (!(ok = warp_wait(&x.s_full[own & 1], (own >> 1) & 1u, &ctl.dead))) break;
        const uint4 valid = *reinterpret_cast<const uint4 *>(ctl.ring.valid[t % kValidRing]);
        const bool masked = tile_masked(p, u, at0, valid);
        const uint32_t s_at = lanes + (t & 1) * 128;
        auto whole = [&] {
          outputs_done(own - 1);
          tc_after();
          return ok;
        };
        if (kSplit) {
          const uint32_t word = ctl.ring.valid[t % kValidRing][part];
          softmax_part<F16, D>(c, mine, masked, seen.x & word, part, s_at, o_at, i == 0, m, l, whole);
        } else if (works) {
          softmax_tile<F16, D>(c, mine, masked, both(seen, valid), s_at, o_at, i == 0, m, l, whole);
        }
        if (!ok) break;
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&x.p_full[own & 1]);
      }
      // the other group goes on with the next unit meanwhile
      if (!ok || !outputs_done(own - 1)) break;
      if constexpr (kSplit) {
        if (!(ok = write_split<E, D, true>(p, u, line.worker, part, lane, o_at, m, l, quarters, &x.meet, met,
                                           &ctl.dead, &ctl.bad)))
          break;
      } else if (works) {
        write_row<E, D, true>(p, u, line.worker, row, n, mine, o_at, m, l,
                              *reinterpret_cast<volatile int *>(&ctl.bad) != 0);
      }
    } while (u.next(p, line));
  } else {
    if constexpr (!kSplit) fewer_regs<kRestRegs4>();
    if (warp < kSplitIssuer) {
    // ------------------------------------------------- operands of the products
    const int maker = warp - 8;
    make_operands<D, kSplitMakers>(p, line, u, maker, lane, wide4_s + Shape::kSplitRaw + maker * Raw4<D>::kWarp,
                                   entries, ctl.ring, &ctl.dead, &ctl.bad);
    } else if (warp == kSplitIssuer) {
    // ------------------------------------------------------------- products
    uint32_t t = 0, own[2] = {0, 0}, units = 0;  // tiles, of each group
    const uint32_t entries_at = smem_u32(entries), q_at = smem_u32(wide4_s);
    auto take = [&](uint32_t e) {  // an entry that is ready
      ok = warp_wait(&ctl.ring.full[e % kRing], (e / kRing) & 1u, &ctl.dead);
      return entries_at + e % kRing * W::kBytes;
    };
    do {
      const int n_tiles = u.i1 - u.i0, g = units & 1;
      auto &x = ctl.group[g];
      const uint32_t base = g ? own[1] : own[0];
      for (int i = 0; i <= n_tiles; ++i) {
        if (i < n_tiles) {  // scores of tile i
          const uint32_t e = 2 * (t + i), k_at = take(e);
          if (!ok || (i == 0 && !(ok = warp_wait(&x.q_full, (units >> 1) & 1u, &ctl.dead)))) break;
          issue_scores<F16, D>(tmem + ((t + i) & 1) * 128, q_at, Shape::kQPanel, k_at);
          issue_commit(&x.s_full[(base + i) & 1]);
          issue_commit(&ctl.ring.empty[e % kRing]);
          if (i + 1 == n_tiles) issue_commit(&x.q_empty);
        }
        if (i > 0) {  // outputs of the tile before
          const uint32_t b = t + i - 1, of = base + i - 1, e = 2 * b + 1, v_at = take(e);
          if (!ok || !(ok = warp_wait(&x.p_full[of & 1], (of >> 1) & 1u, &ctl.dead))) break;
          issue_outputs<F16, D>(tmem + 256 + g * 128, tmem + (b & 1) * 128, v_at, i == 1);
          issue_commit(&x.o_done[of & 1]);
          issue_commit(&ctl.ring.empty[e % kRing]);
        }
      }
      t += n_tiles;
      (g ? own[1] : own[0]) += n_tiles;
      ++units;
    } while (ok && u.next(p, line));
    // nothing is in flight when the tensor memory goes back
    issue_commit(&ctl.drain);
    bar_linger(&ctl.drain, 0u);
    }
  }
  tm_free<kSplitIssuer>(tmem, warp);
  if (!ctl.dead) return;
  void_run<E, D, kThreads>(p, line);
}

namespace {

template <auto kKernel>
cudaError_t start_wide4(int smem, int threads, const AttnParams &p, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  return launch_large(kKernel, done, smem, p.workers, threads, smem, stream, p);
}
template <class E, int D>
cudaError_t start_wide4(const AttnParams &p, cudaStream_t stream) {
  if (p.rows > wide_tile_rows(p.G)) return start_wide4<pair4_kernel<E, D>>(Shape4<D>::kPair, kThreads4, p, stream);
  return p.rows <= 32 ? start_wide4<solo4_kernel<E, D, true>>(Shape4<D>::kSplit, kSplitThreads, p, stream)
                      : start_wide4<solo4_kernel<E, D, false>>(Shape4<D>::kSplit, kThreads4, p, stream);
}

}  // namespace

cudaError_t launch_attention_q4_wide(const AttnParams &p, int dtype, cudaStream_t stream) {
  if (dtype == SPEC_BF16)
    return p.D == 64 ? start_wide4<Bf16, 64>(p, stream) : start_wide4<Bf16, 128>(p, stream);
  return p.D == 64 ? start_wide4<F16, 64>(p, stream) : start_wide4<F16, 128>(p, stream);
}

}  // namespace sv
