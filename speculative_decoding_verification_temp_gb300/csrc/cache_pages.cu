// Operators on the pages of a key-value cache: the new tokens' keys and values
// written (append), the accepted path of a verified tree moved together
// (compact), pages taken and given back (resize), sequences that go on from
// another one's tokens (fork).
//
// Append, compact and the fork's copy move rows in 16-byte pieces and are
// bound by HBM: every moved byte is read once and written once (append of 32
// layers of 32 x 60 tokens, 8 heads of 128 bf16: 72.5 us, 503 MB, 6.9 TB/s; copy
// of 64 partly filled pages of 64 tokens in 32 layers: 71 us).  Resize and the
// fork's bookkeeping are one CTA each, bound by the latency of their few dependent
// global accesses (32 sequences that take and give back 60 tokens on pages of 16: 10
// us for both, 13 with the claims below made always; 256 sequences 30 and 63); they
// take and give pages in a fixed order, so their
// results do not depend on the order in which threads run.
#include <climits>

#include "kv_cache.cuh"

namespace sv {

namespace {

constexpr int kPool = 1024;  // threads of the bookkeeping CTA
constexpr int kPlainShared = 40 * 1024;  // dynamic shared memory that any kernel may use
constexpr int kClaim = -(1 << 30);  // claims on a page are below, counts above

__device__ __forceinline__ uint4 load16(const char *p) {
  return *reinterpret_cast<const uint4 *>(p);
}
__device__ __forceinline__ void store16(char *p, uint4 v) { *reinterpret_cast<uint4 *>(p) = v; }

// Inclusive scan of one value per thread over the CTA; returns the inclusive
// prefix and the total.
__device__ __forceinline__ int block_scan(int v, int *warp_s, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_s[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = lane < warps ? warp_s[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += y;
    }
    warp_s[lane] = w;
  }
  __syncthreads();
  total = warp_s[31];
  return x + (warp ? warp_s[warp - 1] : 0);
}

}  // namespace

// ---------------------------------------------------------------------------
// flags
// ---------------------------------------------------------------------------

__global__ void __launch_bounds__(kThreads)
    kv_flags_kernel(KvSeqs S, KvCache C, bool new_only, int window, int sinks, uint32_t *flags) {
  const int b = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= S.B) return;
  const int ctx = __ldg(S.ctx + b), n = seq_new(S, b);
  uint32_t f = 0u;
  if (S.num_new && __ldg(S.num_new + b) != n) f |= SPEC_FLAG_BAD_LENGTH;
  if (!seq_fits(S, C, ctx, n)) {
    f |= SPEC_FLAG_BAD_LENGTH;
  } else if (n > 0) {
    const int first = new_only ? ctx / C.page_size : 0;
    const int last = (ctx + n - 1) / C.page_size;
    // the first key that a window shows: no new token stands before ctx
    const int shown = window ? ctx - window + 1 : 0;
    for (int i = first + lane; i <= last; i += 32) {
      const int at = i * C.page_size;
      if (at >= sinks && at + C.page_size <= shown) continue;
      if (!page_ok(C, page_at(S, b, i))) f |= SPEC_FLAG_BAD_PAGE;
    }
  }
  f = warp_or(f);
  if (lane == 0) flags[b] = f;
}

cudaError_t launch_kv_flags(const KvSeqs &S, const KvCache &C, bool new_only, int window, int sinks,
                            uint32_t *flags, cudaStream_t stream) {
  kv_flags_kernel<<<(S.B + kWarps - 1) / kWarps, kThreads, 0, stream>>>(S, C, new_only, window,
                                                                         sinks, flags);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// append: slot(ctx + n) of sequence b <- new row n
// ---------------------------------------------------------------------------

// A warp takes one new token: it finds the token's slot once and then copies the
// token's keys and values in the layers blockIdx.y, blockIdx.y + gridDim.y, ...,
// eight 16-byte pieces a lane in flight.
__global__ void __launch_bounds__(kThreads) append_kernel(KvSeqs S, KvCache C, NewRows R) {
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= S.B * S.N) return;
  const int b = t / S.N, n = t - b * S.N;
  const int ctx = __ldg(S.ctx + b), m = seq_new(S, b);
  if (n >= m || !seq_fits(S, C, ctx, m)) return;
  const int at = ctx + n, index = at / C.page_size;
  const int page = page_at(S, b, index);
  if (!page_ok(C, page)) return;
  const int in_page = at - index * C.page_size;
  const int per_row = C.row_bytes / 16, per_token = C.heads * per_row;
  const char *k_src = R.k + b * R.k_seq + n * R.k_token, *v_src = R.v + b * R.v_seq + n * R.v_token;
  char *k_dst = C.k + page * C.k_page + in_page * C.k_token;
  char *v_dst = C.v + page * C.v_page + in_page * C.v_token;
  for (int i0 = lane; i0 < per_token; i0 += 128) {
    long long ks[4], vs[4], kd[4], vd[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * 32, h = i / per_row, c = (i - h * per_row) * 16;
      ks[j] = h * R.k_head + c;
      vs[j] = h * R.v_head + c;
      kd[j] = h * C.k_head + c;
      vd[j] = h * C.v_head + c;
    }
    for (long long layer = blockIdx.y; layer < C.layers; layer += gridDim.y) {
      uint4 x[4], y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i0 + j * 32 < per_token) {
          x[j] = load16(k_src + layer * R.k_layer + ks[j]);
          y[j] = load16(v_src + layer * R.v_layer + vs[j]);
        }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i0 + j * 32 < per_token) {
          store16(k_dst + layer * C.k_layer + kd[j], x[j]);
          store16(v_dst + layer * C.v_layer + vd[j], y[j]);
        }
    }
  }
}

cudaError_t launch_append(const KvSeqs &S, const KvCache &C, const NewRows &R, uint32_t *flags,
                          cudaStream_t stream) {
  if (flags) {
    const cudaError_t e = launch_kv_flags(S, C, true, 0, 0, flags, stream);
    if (e != cudaSuccess) return e;
  }
  if (S.N == 0) return cudaSuccess;
  // two layers a warp where there are enough tokens to fill the card
  const int tokens = S.B * S.N;
  const int split = tokens >= 1024 ? (C.layers + 1) / 2 : C.layers;
  append_kernel<<<dim3((tokens + kWarps - 1) / kWarps, split), kThreads, 0, stream>>>(S, C, R);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// compact: slot(ctx + i) <- slot(ctx + path[i]) for the accepted path
// ---------------------------------------------------------------------------

// A path ascends, so path[i] >= i, and a thread that moves the rows of one
// 16-byte column in ascending order never reads a slot that it has written:
// step i writes slot i, every later source is above it.  Eight sources are
// loaded before their eight targets are stored, for the same reason.  One CTA
// per sequence and layer's keys or values.  Each CTA checks the path and finds
// the byte offsets of the moves' slots, a thread each, into shared memory, so that
// no column looks them up again (32 trees, up to 6 nodes, 32 layers: 8.5 us; 15
// with every column's own look-ups).
struct Move {
  long long from, to;  // from -1: no move
};

__global__ void __launch_bounds__(kThreads)
    compact_kernel(KvSeqs S, KvCache C, const int32_t *path, int width, const int32_t *accepted,
                   int32_t *out_len, uint32_t *flags) {
  extern __shared__ Move move_s[];
  const int b = blockIdx.x, layer = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int ctx = __ldg(S.ctx + b), na = __ldg(accepted + b);
  const int32_t *nodes = path + static_cast<long long>(b) * width;
  const long long s_page = is_v ? C.v_page : C.k_page, s_tok = is_v ? C.v_token : C.k_token;
  const long long s_head = is_v ? C.v_head : C.k_head;
  const int room = S.max_pages * C.page_size;
  uint32_t f = 0u;
  if (na < -1 || na >= width) f |= SPEC_FLAG_BAD_TREE;
  bool ok = na >= 0 && na < width;
  if (ok) {
    auto slot = [&](int at) {
      const int index = at / C.page_size, page = page_at(S, b, index);
      return page_ok(C, page) ? page * s_page + (at - index * C.page_size) * s_tok : -1ll;
    };
    int bad = 0, far = 0, lost = 0;
    for (int i = threadIdx.x; i <= na; i += blockDim.x) {
      const int node = __ldg(nodes + i);
      if (i == 0 ? node != 0 : node <= __ldg(nodes + i - 1)) bad = 1;
      if (ctx < 0 || node < 0 || node >= room - ctx || i >= room - ctx) {
        far = 1;
        continue;
      }
      Move m = {-1, -1};
      if (node != i && i > 0) {
        const long long from = slot(ctx + node), to = slot(ctx + i);
        if (from >= 0 && to >= 0) {
          m = {from, to};
        } else {
          lost = 1;
        }
      } else if (i > 0 && slot(ctx + i) < 0) {
        lost = 1;
      }
      move_s[i] = m;
    }
    bad = __syncthreads_or(bad);
    far = __syncthreads_or(far);
    lost = __syncthreads_or(lost);
    if (bad) {
      f |= SPEC_FLAG_BAD_TREE;
    } else if (far) {
      f |= SPEC_FLAG_BAD_LENGTH;
    } else if (lost) {
      f |= SPEC_FLAG_BAD_PAGE;
    }
    ok = !bad && !far;
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) {
    out_len[b] = ok ? ctx + na + 1 : ctx;
    if (flags) flags[b] = f;
  }
  if (!ok) return;
  char *base = is_v ? C.v + layer * C.v_layer : C.k + layer * C.k_layer;
  const int per_row = C.row_bytes / 16, per_token = C.heads * per_row;
  for (int r = threadIdx.x; r < per_token; r += blockDim.x) {
    const int h = r / per_row;
    char *col = base + h * s_head + (r - h * per_row) * 16;
    for (int i = 1; i <= na; i += 8) {
      uint4 x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j <= na && move_s[i + j].from >= 0) x[j] = load16(col + move_s[i + j].from);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j <= na && move_s[i + j].from >= 0) store16(col + move_s[i + j].to, x[j]);
    }
  }
}

cudaError_t launch_compact(const KvSeqs &S, const KvCache &C, const int32_t *path, int width,
                           const int32_t *accepted, int32_t *out_len, uint32_t *flags,
                           cudaStream_t stream) {
  // a CTA no larger than a token's pieces
  const int per_token = C.heads * (C.row_bytes / 16);
  const int threads = per_token >= kThreads ? kThreads : (per_token + 31) / 32 * 32;
  const dim3 grid(S.B, 2 * C.layers);
  const int smem = width * static_cast<int>(sizeof(Move));
  if (smem > kPlainShared) {
    static std::atomic<uint64_t> done{0};
    return launch_large(compact_kernel, done, kMaxPath * static_cast<int>(sizeof(Move)), grid, threads,
                        smem, stream, S, C, path, width, accepted, out_len, flags);
  }
  compact_kernel<<<grid, threads, smem, stream>>>(S, C, path, width, accepted, out_len, flags);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// resize: each sequence holds ceil(length / page_size) pages
// ---------------------------------------------------------------------------

// One CTA.  Releases first: a reference less for each released entry; a page
// left without references is pushed at its first mention in the order of
// (sequence, entry).  Where a page had several holders, that mention is found with an
// atomicMin of the mention's number, offset below every count, on the page's own
// count, so no scratch is needed.  Then the growing sequences pop theirs in ascending order, as long
// as the pool holds the demand of them and of all before them.
__global__ void __launch_bounds__(kPool, 1)
    resize_kernel(Pool P, const int32_t *length, uint32_t *flags) {
  extern __shared__ int pool_s[];
  __shared__ int warp_s[32];
  int *need_s = pool_s, *have_s = need_s + P.B, *at_s = have_s + P.B;
  uint32_t *flag_s = reinterpret_cast<uint32_t *>(at_s + P.B);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int released = 0, wanted = 0;
  const int top = min(max(__ldcg(P.free_count), 0), P.pages);
  for (int b0 = 0; b0 < P.B; b0 += kPool) {
    const int b = b0 + tid;
    int rel = 0, want = 0;
    if (b < P.B) {
      const int len = length[b];
      int have = P.count[b];
      int need = len / P.page_size + (len % P.page_size > 0);
      uint32_t f = 0u;
      if (len < 0 || need > P.max_pages || have < 0 || have > P.max_pages) {
        f = SPEC_FLAG_BAD_LENGTH;
        need = have = min(max(have, 0), P.max_pages);
      }
      need_s[b] = need;
      have_s[b] = have;
      flag_s[b] = f;
      rel = max(have - need, 0);
      want = max(need - have, 0);
    }
    int total;
    const int upto = block_scan(rel, warp_s, total);
    if (b < P.B) at_s[b] = released + upto - rel;
    released += total;
    block_scan(want, warp_s, total);
    wanted += total;
  }
  __syncthreads();
  int filled = top;
  if (released > 0) {  // the same for every thread
    int *freed_s = reinterpret_cast<int *>(flag_s + P.B);
    int shared = 0;
    for (int b = warp; b < P.B; b += kPool / 32) {
      const int need = need_s[b], have = have_s[b];
      const int32_t *row = P.table + static_cast<long long>(b) * P.ld_table;
      bool bad = false;
      int n = 0;
      for (int i0 = need; i0 < have; i0 += 32) {
        const int i = i0 + lane, page = i < have ? row[i] : -1;
        const bool good = static_cast<unsigned>(page) < static_cast<unsigned>(P.pages);
        const int held = good ? atomicSub(P.refs + page, 1) : 0;
        bad |= i < have && held <= 0;
        shared |= good && held != 1;
        n += __popc(__ballot_sync(0xFFFFFFFFu, held == 1));
      }
      bad = __any_sync(0xFFFFFFFFu, bad);
      if (lane == 0) {
        if (bad) flag_s[b] |= SPEC_FLAG_BAD_PAGE;
        freed_s[b] = n;
      }
    }
    // where every mention found one holder, every page was mentioned once and is
    // free now: there is nothing to claim
    const bool claims = __syncthreads_or(shared);
    // whether this mention frees the page
    auto mine = [&](int page, int mention) {
      return static_cast<unsigned>(page) < static_cast<unsigned>(P.pages) &&
             (!claims || __ldcg(P.refs + page) == INT_MIN + mention);
    };
    if (claims) {
      for (int b = warp; b < P.B; b += kPool / 32) {
        const int need = need_s[b], have = have_s[b], base = at_s[b];
        const int32_t *row = P.table + static_cast<long long>(b) * P.ld_table;
        for (int i = need + lane; i < have; i += 32) {
          const int page = row[i];
          if (static_cast<unsigned>(page) >= static_cast<unsigned>(P.pages)) continue;
          const int refs = __ldcg(P.refs + page);
          if (refs == 0 || refs < kClaim) atomicMin(P.refs + page, INT_MIN + base + i - need);
        }
      }
      __syncthreads();
      // pages freed by each sequence
      for (int b = warp; b < P.B; b += kPool / 32) {
        const int need = need_s[b], have = have_s[b], base = at_s[b];
        const int32_t *row = P.table + static_cast<long long>(b) * P.ld_table;
        int n = 0;
        for (int i0 = need; i0 < have; i0 += 32) {
          const int i = i0 + lane;
          n += __popc(__ballot_sync(0xFFFFFFFFu, i < have && mine(row[i], base + i - need)));
        }
        if (lane == 0) freed_s[b] = n;
      }
      __syncthreads();
    }
    // ... and by those before it
    int freed = 0;
    for (int b0 = 0; b0 < P.B; b0 += kPool) {
      const int b = b0 + tid, n = b < P.B ? freed_s[b] : 0;
      int total;
      const int upto = block_scan(n, warp_s, total);
      if (b < P.B) freed_s[b] = freed + upto - n;
      freed += total;
    }
    __syncthreads();
    for (int b = warp; b < P.B; b += kPool / 32) {
      const int need = need_s[b], have = have_s[b], base = at_s[b];
      int32_t *row = P.table + static_cast<long long>(b) * P.ld_table;
      int place = top + freed_s[b];
      for (int i0 = need; i0 < have; i0 += 32) {
        const int i = i0 + lane;
        const int page = i < have ? row[i] : -1;
        const bool push = i < have && mine(page, base + i - need);
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, push);
        // a list that is too long already was not made by these operators
        if (push) {
          const int p = place + __popc(who & ((1u << lane) - 1u));
          if (p < P.pages) P.free_list[p] = page;
        }
        place += __popc(who);
        if (!claims && i < have) row[i] = -1;
      }
    }
    __syncthreads();
    if (claims) {
      for (int b = warp; b < P.B; b += kPool / 32) {
        const int need = need_s[b], have = have_s[b];
        int32_t *row = P.table + static_cast<long long>(b) * P.ld_table;
        for (int i = need + lane; i < have; i += 32) {
          const int page = row[i];
          if (static_cast<unsigned>(page) < static_cast<unsigned>(P.pages) &&
              __ldcg(P.refs + page) < kClaim)
            P.refs[page] = 0;  // every mention of the page writes the same value
          row[i] = -1;
        }
      }
    }
    filled = min(top + freed, P.pages);
    __syncthreads();
  }
  int taken = 0;
  if (wanted > 0) {
    int before = 0;
    for (int b0 = 0; b0 < P.B; b0 += kPool) {
      const int b = b0 + tid;
      const int want = b < P.B ? max(need_s[b] - have_s[b], 0) : 0;
      int demand, given;
      const int upto = before + block_scan(want, warp_s, demand);
      const bool served = want > 0 && upto <= filled;
      block_scan(served ? want : 0, warp_s, given);
      if (b < P.B) at_s[b] = upto - want;
      if (want > 0 && !served) {
        flag_s[b] |= SPEC_FLAG_NO_PAGES;
        need_s[b] = have_s[b];
      }
      before += demand;
      taken += given;
    }
    __syncthreads();
    for (int b = warp; b < P.B; b += kPool / 32) {
      if (need_s[b] <= have_s[b]) continue;
      const int have = have_s[b], want = need_s[b] - have, first = filled - 1 - at_s[b];
      int32_t *row = P.table + static_cast<long long>(b) * P.ld_table;
      bool bad = false;
      for (int j = lane; j < want; j += 32) {
        const int page = __ldcg(P.free_list + first - j);
        P.free_list[first - j] = -1;
        const bool good = static_cast<unsigned>(page) < static_cast<unsigned>(P.pages);
        row[have + j] = good ? page : -1;
        if (good) P.refs[page] = 1;
        bad |= !good;
      }
      if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) flag_s[b] |= SPEC_FLAG_BAD_PAGE;
    }
  }
  __syncthreads();
  for (int b = tid; b < P.B; b += kPool) {
    P.count[b] = need_s[b];
    if (flags) flags[b] = flag_s[b];
  }
  if (tid == 0) *P.free_count = filled - taken;
}

cudaError_t launch_resize(const Pool &P, const int32_t *length, uint32_t *flags,
                          cudaStream_t stream) {
  constexpr int kPerSeq = 5 * static_cast<int>(sizeof(int));
  const int smem = P.B * kPerSeq;
  if (smem > kPlainShared) {
    static std::atomic<uint64_t> done{0};
    return launch_large(resize_kernel, done, kMaxSeqs * kPerSeq, 1, kPool, smem, stream, P, length,
                        flags);
  }
  resize_kernel<<<1, kPool, smem, stream>>>(P, length, flags);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// fork: sequence dst[f] goes on from the tokens of sequence src[f]
// ---------------------------------------------------------------------------

struct PageCopy {
  int from, to, rows;
};

// One CTA.  Every fork reads its source before any row is written.  Of the
// forks that name one target the lowest takes it (an atomicMin of the fork's
// number on the target's page count, which is zero); the pages for the last,
// partly filled ones are popped in the order of the forks.
__global__ void __launch_bounds__(kPool, 1)
    fork_plan_kernel(Pool P, int32_t *ctx, const int32_t *src, const int32_t *dst, int F,
                     PageCopy *copies, uint32_t *flags) {
  extern __shared__ int pool_s[];
  __shared__ int warp_s[32];
  int *len_s = pool_s, *rank_s = len_s + F;  // length -1: the fork does nothing
  uint32_t *flag_s = reinterpret_cast<uint32_t *>(rank_s + F);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int top = min(max(__ldcg(P.free_count), 0), P.pages);
  for (int f = tid; f < F; f += kPool) {
    const int s = src[f], d = dst[f];
    int len = -1;
    uint32_t fl = 0u;
    if (s < 0 || s >= P.B || d < 0 || d >= P.B) {
      fl = SPEC_FLAG_BAD_SEQUENCE;
    } else {
      len = __ldcg(ctx + s);
      const int need = len / P.page_size + (len % P.page_size > 0);
      if (len < 0 || need > P.max_pages || __ldcg(P.count + s) < need) {
        fl = SPEC_FLAG_BAD_LENGTH;
        len = -1;
      } else if (__ldcg(P.count + d) != 0) {
        fl = SPEC_FLAG_BAD_SEQUENCE;
        len = -1;
      }
    }
    len_s[f] = len;
    flag_s[f] = fl;
  }
  __syncthreads();
  for (int f = tid; f < F; f += kPool)
    if (len_s[f] >= 0) atomicMin(P.count + dst[f], INT_MIN + f);
  __syncthreads();
  int before = 0, taken = 0;
  for (int f0 = 0; f0 < F; f0 += kPool) {
    const int f = f0 + tid;
    int part = 0;
    if (f < F && len_s[f] >= 0) {
      if (__ldcg(P.count + dst[f]) != INT_MIN + f) {
        flag_s[f] = SPEC_FLAG_BAD_SEQUENCE;
        len_s[f] = -1;
      } else {
        part = len_s[f] % P.page_size > 0;
      }
    }
    int demand, given;
    const int upto = before + block_scan(part, warp_s, demand);
    const bool served = part && upto <= top;
    block_scan(served, warp_s, given);
    if (f < F) rank_s[f] = upto - part;
    if (part && !served) {
      flag_s[f] = SPEC_FLAG_NO_PAGES;
      len_s[f] = -2;  // owns its target, whose count goes back to zero
    }
    before += demand;
    taken += given;
  }
  __syncthreads();
  for (int f = warp; f < F; f += kPool / 32) {
    const int len = len_s[f];
    PageCopy copy = {0, 0, 0};
    if (len == -2 && lane == 0) P.count[dst[f]] = 0;
    if (len >= 0) {
      const int s = src[f], d = dst[f];
      const int full = len / P.page_size, rest = len - full * P.page_size;
      const int32_t *from = P.table + static_cast<long long>(s) * P.ld_table;
      int32_t *to = P.table + static_cast<long long>(d) * P.ld_table;
      int fresh = -1;
      bool bad = false;
      if (rest > 0) {
        const int at = top - 1 - rank_s[f];
        fresh = __ldcg(P.free_list + at);
        const int old = from[full];
        __syncwarp();
        const bool good = static_cast<unsigned>(fresh) < static_cast<unsigned>(P.pages);
        const bool old_good = static_cast<unsigned>(old) < static_cast<unsigned>(P.pages);
        if (good && old_good) copy = {old, fresh, rest};
        if (!good) fresh = -1;
        bad = !good || !old_good;
        if (lane == 0) {
          P.free_list[at] = -1;
          if (good) P.refs[fresh] = 1;
        }
      }
      for (int i = lane; i < P.max_pages; i += 32) {
        int page = -1;
        if (i < full) {
          page = from[i];
          if (static_cast<unsigned>(page) < static_cast<unsigned>(P.pages)) {
            atomicAdd(P.refs + page, 1);
          } else {
            page = -1;
            bad = true;
          }
        } else if (i == full && rest > 0) {
          page = fresh;
        }
        to[i] = page;
      }
      bad = __any_sync(0xFFFFFFFFu, bad);
      if (lane == 0) {
        P.count[d] = full + (rest > 0);
        ctx[d] = len;
        if (bad) flag_s[f] |= SPEC_FLAG_BAD_PAGE;
      }
    }
    if (lane == 0) {
      copies[f] = copy;
      if (flags) flags[f] = flag_s[f];
    }
  }
  if (tid == 0) *P.free_count = top - taken;
}

// The rows of the partly filled pages: one CTA per fork and layer's keys or
// values.
__global__ void __launch_bounds__(kThreads)
    page_copy_kernel(KvCache C, const PageCopy *copies) {
  const int layer = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  char *base = is_v ? C.v + layer * C.v_layer : C.k + layer * C.k_layer;
  const long long s_page = is_v ? C.v_page : C.k_page, s_tok = is_v ? C.v_token : C.k_token;
  const long long s_head = is_v ? C.v_head : C.k_head;
  const int per_row = C.row_bytes / 16, per_token = C.heads * per_row;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PageCopy copy = copies[blockIdx.x];
  const char *from = base + copy.from * s_page;
  char *to = base + copy.to * s_page;
  const int pieces = copy.rows * per_token;
  for (int i0 = threadIdx.x; i0 < pieces; i0 += 4 * kThreads) {
    uint4 x[4];
    long long off[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * kThreads;
      const int t = i / per_token, r = i - t * per_token;
      off[j] = t * s_tok + (r / per_row) * s_head + (r % per_row) * 16;
      if (i < pieces) x[j] = load16(from + off[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + j * kThreads < pieces) store16(to + off[j], x[j]);
  }
}

size_t fork_workspace_bytes(int F) { return static_cast<size_t>(F) * sizeof(PageCopy); }

cudaError_t launch_fork(const Pool &P, const KvCache &C, int32_t *ctx, const int32_t *src,
                        const int32_t *dst, int F, void *workspace, uint32_t *flags,
                        cudaStream_t stream) {
  PageCopy *copies = static_cast<PageCopy *>(workspace);
  constexpr int kPerFork = 3 * static_cast<int>(sizeof(int));
  const int smem = F * kPerFork;
  cudaError_t e;
  if (smem > kPlainShared) {
    static std::atomic<uint64_t> done{0};
    e = launch_large(fork_plan_kernel, done, kMaxSeqs * kPerFork, 1, kPool, smem, stream, P, ctx, src,
                     dst, F, copies, flags);
  } else {
    fork_plan_kernel<<<1, kPool, smem, stream>>>(P, ctx, src, dst, F, copies, flags);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  return launch_behind(page_copy_kernel, dim3(F, 2 * C.layers), kThreads, 0, stream, C,
                       static_cast<const PageCopy *>(copies));
}

}  // namespace sv
