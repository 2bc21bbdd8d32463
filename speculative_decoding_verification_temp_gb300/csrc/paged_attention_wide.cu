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

#include "paged_attention_wide.cuh"

namespace sv {

namespace {

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
                               o_at + lanes, i == 0, m, l, [] { return true; });
          } else if (works) {
            softmax_tile<E, D>(p.scale_log2, mine, masked, both(seen, valid), s_at + lanes,
                               o_at + lanes, i == 0, m, l, [] { return true; });
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
          if (sent == 0) first_wait(&st.full[0], p.first_wait, &ctl.dead);
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
                             s_at, o_at, i == 0, m, l, [] { return true; });
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
        if (!values && sent == 0) first_wait(&ctl.full[0], p.first_wait, &ctl.dead);
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
