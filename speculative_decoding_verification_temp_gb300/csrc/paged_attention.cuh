// Attention of new tokens over a paged key-value cache: what its kernels share.
//
// The rows of a (sequence, head of the cache) are its new tokens times the
// group of query heads that read this head: row r is token r / G, query head
// h * G + r % G.  A unit is a tile of R rows with all the keys that one of them
// may see, cut into tiles of T keys.  The units' key tiles, laid end to end
// (sequences, then heads, then row tiles; a unit's end takes some places more,
// for what a unit costs beside its keys), are one line of work that is cut into
// equal runs, one per worker (a CTA, or one of its two streams), whatever the
// lengths of the sequences are: a worker's run holds whole units, which it
// finishes, and at most one unit's end and one unit's beginning, which it leaves
// as partial results (running maximum, sum and unnormalised output of each row).
// A second kernel joins the partial results of each unit that was cut, in the
// order of its keys, so results do not depend on timing.  The line is laid out
// on the device from the lengths, so a captured launch follows lengths that
// change.
//
// A piece costs beside its keys what a unit does, and the join besides.  Where the
// page table or the window keeps all units short (`whole`), a worker takes the whole
// of those that begin in its run, and there is no join.
//
// Where a sequence has several row tiles with the same keys (row_lines of them),
// each has a line and an equal share of the workers of its own: neighbouring
// workers then go through the same keys at the same time, and HBM is read once
// for all of them instead of once for each.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_cache.cuh"

namespace sv {

struct AttnParams {
  const char *q;
  long long q_seq, q_token, q_head;  // bytes
  KvCache C;
  KvSeqs S;
  const uint64_t *mask;
  long long mask_seq;
  int words;
  const int32_t *position;
  long long position_seq;
  int G, D;
  float scale, scale_log2;
  int window, sinks;
  void *out;
  float *lse;
  uint32_t *flags;
  float *part;  // partial results, two slots per worker
  struct JoinDesc *join;
  int workers, rows, tile_log2;  // at most; R; T as a power of two
  int unit_cost;                 // places on the line behind a unit's key tiles
  int row_lines;                 // 1: all row tiles on one line
  bool whole;                    // units are not cut, and not joined
  long long first_wait;          // cycles of a run's first wait (spec_set_wait_limit)
};

// A cut unit, written by the worker that holds its first cut; its pieces are
// those of its line's worker before it .. pieces_end.  pieces_end -1: no unit's cuts
// start here.
struct JoinDesc {
  int b, h, r0, rows, pieces_end;
};

size_t attention_workspace_bytes(int N, int G, int D, int dtype);
cudaError_t launch_attention(AttnParams &p, int dtype, void *workspace, cudaStream_t stream);
// The form on tensor memory: one or two tiles of wide_tile_rows(G) rows per unit
// (p.rows), head_dim 64 or 128, 16-bit types.  wide_maps: false where the
// tensors cannot be described to TMA.
struct WideMaps {
  CUtensorMap k, v, q;
  // coordinate of a box: page * k_page + head * k_head + token * k_token, ...
  int k_page, k_head, k_token, v_page, v_head, v_token, q_seq, q_head;
};
// Rows of a tile: whole tokens, at most 128 rows.
inline int wide_tile_rows(int G) { return 128 / G * G; }
bool wide_maps(const AttnParams &p, int dtype, WideMaps *maps);
// Cycles that spec_set_wait_limit allows a first wait.
long long first_wait_cycles();
cudaError_t launch_attention_wide(const AttnParams &p, const WideMaps &maps, int dtype,
                                  cudaStream_t stream);

// The keys that the rows [r0, r0 + R) of sequence b may see: tiles
// [0, sink_tiles) and then `lo` and those behind it; at least one tile, which
// may hold no visible key.
struct KeyRange {
  int ctx, n_new;   // n_new: new tokens, 0 where the sequence does not fit
  int end;          // keys at or behind it are seen by no row
  int all;          // keys before it are seen by every row, but for the window
  int first;        // keys before it are seen by no row, but for the sinks
  int sink_tiles, lo, count;
};

__device__ __forceinline__ KeyRange key_range(const AttnParams &p, int ctx, int n_new, bool fits,
                                              int r0) {
  const int round = (1 << p.tile_log2) - 1;
  KeyRange k;
  k.ctx = ctx;
  k.n_new = n_new;
  k.end = k.all = k.first = 0;
  if (fits) {
    const int n_lo = r0 == 0 ? 0 : r0 / p.G;
    const int n_hi = r0 + p.rows >= n_new * p.G ? n_new - 1 : (r0 + p.rows - 1) / p.G;
    k.end = p.mask ? ctx + n_new : ctx + n_hi + 1;
    k.all = p.mask ? ctx : ctx + n_lo + 1;
    if (p.window) k.first = max(0, (p.mask || p.position ? ctx : ctx + n_lo) - p.window + 1);
  }
  k.lo = k.first >> p.tile_log2;
  k.sink_tiles = p.window ? min((min(p.sinks, k.end) + round) >> p.tile_log2, k.lo) : 0;
  k.count = max(1, k.sink_tiles + ((k.end + round) >> p.tile_log2) - k.lo);
  return k;
}

__device__ __forceinline__ int key_tile(const KeyRange &k, int i) {
  return i < k.sink_tiles ? i : k.lo + i - k.sink_tiles;
}

// Quotient of two whole numbers that are mostly small.
__device__ __forceinline__ long long div_small(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// Places of one head of a sequence.
__device__ __forceinline__ long long head_work(const AttnParams &p, int ctx, int n_new, bool fits,
                                               int line) {
  const int rows = n_new * p.G;
  if (rows <= line * p.rows) return 0;
  if (p.row_lines > 1)
    return key_range(p, ctx, n_new, fits, line * p.rows).count + p.unit_cost;
  if (rows <= p.rows || p.mask || !fits) {  // its row tiles have the same keys
    const int tiles = rows <= p.rows ? 1 : (rows + p.rows - 1) / p.rows;
    return static_cast<long long>(tiles) * (key_range(p, ctx, n_new, fits, 0).count + p.unit_cost);
  }
  long long w = 0;
  for (int r0 = 0; r0 < rows; r0 += p.rows)
    w += key_range(p, ctx, n_new, fits, r0).count + p.unit_cost;
  return w;
}

// A worker's run.  The line's places are dealt out in order, one more to each of
// the first `more` workers.
struct Line {
  long long w0, w1;     // empty: no work
  long long per, more;
  int worker, line;     // the line is `worker` modulo row_lines,
  int turn, turns;      // its run on it the turn-th of those with work
  int b;                // the sequence that holds w0
  long long in_seq;     // w0 within it

  __device__ __forceinline__ long long start_of(long long w) const { return w * per + min(w, more); }
  __device__ __forceinline__ long long turn_of(long long place) const {
    const long long cut = more * (per + 1);
    return place < cut ? div_small(place, per + 1) : more + div_small(place - cut, per);
  }
};

// Shared memory that find_runs works in.
template <int kT, int kW>
struct RunScratch {
  long long sums[kT / 32];
  long long found[kW][2];
};

// The runs of kW workers of a CTA (first, first + step, ...), by all its kT
// threads.
template <int kT, int kW>
__device__ __forceinline__ void find_runs(const AttnParams &p, RunScratch<kT, kW> &x, int first,
                                          int step, Line (&L)[kW]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // (with more than one line, of one worker)
  const int line = p.row_lines == 1 ? 0 : first % p.row_lines;
  const int chunk = (p.S.B + kT - 1) / kT;
  const int b0 = min(tid * chunk, p.S.B), b1 = min(b0 + chunk, p.S.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int ctx = __ldg(p.S.ctx + b), n = seq_new(p.S, b);
    mine += p.C.heads * head_work(p, ctx, n, seq_fits(p.S, p.C, ctx, n), line);
  }
  long long before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, before, o);
    if (lane >= o) before += y;
  }
  if (lane == 31) x.sums[warp] = before;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kT / 32; ++w) {
    const long long v = x.sums[w];
    if (w < warp) before += v;
    total += v;
  }
  before -= mine;
  const int most = p.row_lines == 1 ? p.workers : p.workers / p.row_lines;
  const int turns = total < most ? (total > 0 ? static_cast<int>(total) : 1) : most;
  const long long per = div_small(total, turns);
#pragma unroll
  for (int i = 0; i < kW; ++i) {
    L[i].per = per;
    L[i].more = total - per * turns;
    L[i].turns = turns;
    L[i].worker = first + i * step;
    L[i].line = line;
    L[i].turn = p.row_lines == 1 ? L[i].worker : L[i].worker / p.row_lines;
    const bool busy = total > 0 && L[i].turn < turns;
    L[i].w0 = busy ? L[i].start_of(L[i].turn) : 0;
    L[i].w1 = busy ? L[i].start_of(L[i].turn + 1ll) : 0;
    if (busy && before <= L[i].w0 && L[i].w0 < before + mine) {
      long long at = before;
      for (int b = b0; b < b1; ++b) {
        const int ctx = __ldg(p.S.ctx + b), n = seq_new(p.S, b);
        const long long w = p.C.heads * head_work(p, ctx, n, seq_fits(p.S, p.C, ctx, n), line);
        if (L[i].w0 < at + w) {
          x.found[i][0] = b;
          x.found[i][1] = L[i].w0 - at;
          break;
        }
        at += w;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kW; ++i) {
    const bool busy = L[i].w0 < L[i].w1;
    L[i].b = busy ? static_cast<int>(x.found[i][0]) : 0;
    L[i].in_seq = busy ? x.found[i][1] : 0;
  }
}

// Walks the units of a run.
struct UnitWalk {
  int b, h, r0;
  KeyRange k;
  bool fits;
  long long a;    // the unit's first place on the line
  int i0, i1;     // the run's tiles of the unit

  __device__ __forceinline__ void load_seq(const AttnParams &p) {
    k.ctx = __ldg(p.S.ctx + b);
    k.n_new = seq_new(p.S, b);
    fits = seq_fits(p.S, p.C, k.ctx, k.n_new);
  }
  // The first unit; false: the run has no tiles.
  __device__ __forceinline__ bool start(const AttnParams &p, const Line &L) {
    if (L.w0 == L.w1) return false;
    b = L.b;
    load_seq(p);
    const long long per_head = head_work(p, k.ctx, k.n_new, fits, L.line);
    h = static_cast<int>(div_small(L.in_seq, per_head));
    long long left = L.in_seq - h * per_head;
    for (r0 = L.line * p.rows;; r0 += p.rows) {
      k = key_range(p, k.ctx, k.n_new, fits, r0);
      if (left < k.count + p.unit_cost) break;
      left -= k.count + p.unit_cost;
    }
    a = L.w0 - left;
    i0 = static_cast<int>(p.whole && left > 0 ? k.count : left);
    i1 = end_of(p, L);
    return i0 < i1 || next(p, L);
  }
  // The run's end in the unit.
  __device__ __forceinline__ int end_of(const AttnParams &p, const Line &L) const {
    return p.whole ? k.count : static_cast<int>(min(static_cast<long long>(k.count), L.w1 - a));
  }
  // The next unit; false: the run ends before it.
  __device__ __forceinline__ bool next(const AttnParams &p, const Line &L) {
    a += k.count + p.unit_cost;
    if (a >= L.w1) return false;
    r0 += p.rows;
    if (p.row_lines > 1 || r0 >= k.n_new * p.G) {
      r0 = L.line * p.rows;
      if (++h == p.C.heads) {
        h = 0;
        do {
          ++b;
          load_seq(p);
        } while (k.n_new * p.G <= r0);
      }
    }
    k = key_range(p, k.ctx, k.n_new, fits, r0);
    i0 = 0;
    i1 = end_of(p, L);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return i0 == 0 && i1 == k.count; }
  // Rows of the unit that exist.
  __device__ __forceinline__ int live_rows(const AttnParams &p) const {
    return min(p.rows, k.n_new * p.G - r0);
  }
};

// Slot of the workspace for a worker's piece of a cut unit.
__device__ __forceinline__ int piece_slot(const UnitWalk &u, int worker) {
  return 2 * worker + (u.i0 > 0 ? 0 : 1);
}
// A slot: m of each row, l of each row, padding to 32 bytes, the rows' outputs.
__host__ __device__ __forceinline__ size_t slot_stats(int R) { return (2 * R + 7) / 8 * 8; }
__host__ __device__ __forceinline__ size_t slot_floats(int R, int D) {
  return (slot_stats(R) + static_cast<size_t>(R) * D + 7) / 8 * 8;
}

// Writes a worker's join descriptor: the unit that its first tile cuts, if no
// worker before it cuts that unit.  u: its first unit, or NULL.
__device__ __forceinline__ void write_join(const AttnParams &p, const Line &L, const UnitWalk *u) {
  if (L.worker >= p.workers) return;
  JoinDesc d = {0, 0, 0, 0, -1};
  if (u && u->i0 > 0 && L.start_of(L.turn - 1ll) <= u->a) {
    d.b = u->b;
    d.h = u->h;
    d.r0 = u->r0;
    d.rows = u->live_rows(p);
    d.pieces_end =
        static_cast<int>(L.turn_of(u->a + u->k.count - 1)) * p.row_lines + L.line;
  }
  p.join[L.worker] = d;
}

// The place of new token m behind the context, for windows.
__device__ __forceinline__ int clamp_pos(const AttnParams &p, int b, int m) {
  if (!p.position) return m;
  return min(max(__ldg(p.position + static_cast<long long>(b) * p.position_seq + m), 0),
             p.S.N - 1);
}
// Whether new token n sees the key at index `at` of the sequence.
__device__ __forceinline__ bool sees(const AttnParams &p, const KeyRange &k, int b, int n, int at) {
  int place = at;
  if (at >= k.ctx) {
    const int m = at - k.ctx;
    if (m >= k.n_new) return false;
    if (p.mask) {
      const uint64_t w = __ldg(reinterpret_cast<const unsigned long long *>(p.mask) +
                               static_cast<long long>(b) * p.mask_seq +
                               static_cast<long long>(n) * p.words + (m >> 6));
      if (!((w >> (m & 63)) & 1ull)) return false;
    } else if (m > n) {
      return false;
    }
    if (p.window) place = k.ctx + clamp_pos(p, b, m);
  }
  if (p.window && place >= p.sinks && k.ctx + clamp_pos(p, b, n) - place >= p.window) return false;
  return true;
}

// Whether every row of the unit sees all of the keys [at, at + n).
__device__ __forceinline__ bool all_seen(const AttnParams &p, const KeyRange &k, int at, int n) {
  if (at + n > k.all) return false;
  if (!p.window) return true;
  if (at + n > k.ctx) return false;
  // before the last place that a new token can have
  return at + n <= p.sinks || at > k.ctx + p.S.N - 1 - p.window;
}

// ---------------------------------------------------------------------------
// element types
// ---------------------------------------------------------------------------

struct Bf16 {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float to(T x) { return __bfloat162float(x); }
  static __device__ __forceinline__ T from(float x) { return __float2bfloat16_rn(x); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
  }
  static constexpr uint32_t kExp = 0x7F80u;  // all ones: infinity or NaN
  static constexpr bool kNarrow = false;     // exponents as float32
};
struct F16 {
  using T = __half;
  static __device__ __forceinline__ float to(T x) { return __half2float(x); }
  static __device__ __forceinline__ T from(float x) { return __float2half_rn(x); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
  }
  static constexpr uint32_t kExp = 0x7C00u;
  static constexpr bool kNarrow = true;  // 2^-24 to 2^15
};

// Four outputs of one row: stored as the cache's type.
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(Bf16::pack(v.x, v.y), Bf16::pack(v.z, v.w));
}
__device__ __forceinline__ void store4(__half *p, float4 v) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(F16::pack(v.x, v.y), F16::pack(v.z, v.w));
}
__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_f32(__half x) { return __half2float(x); }

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes from global to shared memory, or 16 zero bytes.
__device__ __forceinline__ void copy16(uint32_t to, const char *from, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int n>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// A 32-bit word of two 16-bit values with infinities and NaNs set to zero.
template <class E>
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t v) {
  if ((v & E::kExp) == E::kExp) v &= 0xFFFF0000u;
  if (((v >> 16) & E::kExp) == E::kExp) v &= 0xFFFFu;
  return v;
}

// Address of row r of a unit in [B, N, Hq] rows.
__device__ __forceinline__ long long out_row(const AttnParams &p, int b, int h, int r) {
  const int n = r / p.G, g = r - n * p.G;
  return (static_cast<long long>(b) * p.S.N + n) * (p.C.heads * p.G) + h * p.G + g;
}

// ln of the weights' sum, from m and l of a row (base 2).
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

// Keys whose values hold infinities or NaNs, in slices that some row does not
// see whole: their values enter the products as zero where some row does not
// see them, so that 0 * inf does not reach that row.  What they add to the rows
// that do is an infinity or a NaN whatever the weight, and is added here: four
// outputs of token n, from the slices (kSlice keys) of tiles [i0, i1).  Reached
// only when such a value was found.
template <class TE, int kSlice>
static __device__ __noinline__ float4 nonfinite_values(const AttnParams &p, const UnitWalk u, int n,
                                                int d, float4 acc) {
  float *a = reinterpret_cast<float *>(&acc);
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
        const TE *v = reinterpret_cast<const TE *>(p.C.v + page * p.C.v_page +
                                                   (at - index * p.C.page_size) * p.C.v_token +
                                                   u.h * p.C.v_head);
        for (int j = 0; j < 4; ++j) {
          const float x = as_f32(v[d + j]);
          if (!isfinite(x)) a[j] += x;
        }
      }
    }
  }
  return acc;
}

}  // namespace sv
