// New tokens' rows on their way into the paged cache and out of it: queries and
// keys rotated by their positions, keys and values written to their pages as they
// are or as 4-bit rows (q4.cuh), and read back.
//
// Rotation: a pair (a, b) of a head's values becomes (a cos t - b sin t, a sin t +
// b cos t), t = position * frequency.  Far positions times frequencies lose their
// angle in float32, and float64 is slow here, so a frequency becomes the fraction of
// a turn per token in 64-bit fixed point once per thread; an integer product that
// wraps is then the angle itself, off by 2^-54 turns per token of position, and
// sine and cosine see a float32 in [-1/2, 1/2] turns.  A CTA takes a batch of tokens
// (kRotThreads / pairs at most): one thread per (token, pair) finds the angle, and all
// of the tokens' heads use it from shared memory.
//
// All kernels here are bound by HBM: rows are read once and written once, in 16-byte
// pieces, a thread holding both pieces of its pairs, so that queries may be rotated in
// place.
#include <algorithm>

#include "paged_attention.cuh"
#include "q4.cuh"
#include "rotary.cuh"

namespace sv {

namespace {

constexpr int kRotThreads = 256;

struct F32 {
  using T = float;
  static __device__ __forceinline__ float to(T x) { return x; }
  static __device__ __forceinline__ T from(float x) { return x; }
};

// 16 bytes of a row as float32.
template <class E>
struct Piece {
  static constexpr int kN = 16 / sizeof(typename E::T);
  float x[kN];
  __device__ __forceinline__ void load(const char *p) { set(*reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void set(const uint4 &v) {
    const typename E::T *t = reinterpret_cast<const typename E::T *>(&v);
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] = E::to(t[i]);
  }
  __device__ __forceinline__ uint4 get() const {
    uint4 v;
    typename E::T *t = reinterpret_cast<typename E::T *>(&v);
#pragma unroll
    for (int i = 0; i < kN; ++i) t[i] = E::from(x[i]);
    return v;
  }
};

// A thread's frequency as turns per token, in units of 2^-64 turns.
__device__ __forceinline__ unsigned long long turn_of(double frequency) {
  const double r = frequency * 0.15915494309189533577;  // 1 / (2 pi)
  return static_cast<unsigned long long>(
      static_cast<long long>(__double2ull_rd((r - floor(r)) * 18446744073709551616.0)));
}

// cos and sin of every (token of the batch, pair), by the whole CTA; place(i): the
// position of token i of the batch.  Ends with a barrier.
template <class Place>
__device__ __forceinline__ void find_angles(const Rotation &r, int tokens, Place place, float2 *cs) {
  // pairs <= kRotThreads: a thread keeps its pair
  const int per = kRotThreads / r.pairs, pair = threadIdx.x % r.pairs;
  const int first = threadIdx.x / r.pairs;
  if (first < per && first < tokens) {
    const double f = __ldg(r.frequency + pair);
    const unsigned long long turn = turn_of(f);
    for (int i = first; i < tokens; i += per) {
      const long long at = place(i);
      // two's complement: the fraction nearest to zero
      const long long fraction = static_cast<long long>(turn * static_cast<unsigned long long>(at));
      float s, c;
      // fraction * 2^-64 turns are fraction * 2^-63 half turns
      sincospif(static_cast<float>(fraction) * 1.0842021724855044e-19f, &s, &c);
      if (!isfinite(f)) s = c = __int_as_float(0x7FC00000);
      cs[i * r.pairs + pair] = make_float2(c * r.amplitude, (r.inverse ? -s : s) * r.amplitude);
    }
  }
  __syncthreads();
}

__device__ __forceinline__ void turn(float &a, float &b, float2 cs) {
  const float x = fmaf(a, cs.x, -(b * cs.y));
  b = fmaf(a, cs.y, b * cs.x);
  a = x;
}

// One row rotated, by the `lanes` threads of which this is the lane-th.  kVector:
// the pairs' halves begin at 16-byte pieces.
template <class E, bool kVector>
__device__ __forceinline__ void rotate_row(const char *from, char *to, int D, const Rotation &r,
                                           const float2 *cs, int lane, int lanes) {
  using T = typename E::T;
  constexpr int kN = Piece<E>::kN;
  if constexpr (kVector) {
    const int pieces = D / kN;
    if (r.interleaved) {
      const int turned = 2 * r.pairs / kN;
      for (int i = lane; i < pieces; i += lanes) {
        uint4 v = *reinterpret_cast<const uint4 *>(from + i * 16);
        if (i < turned) {
          Piece<E> p;
          p.set(v);
#pragma unroll
          for (int e = 0; e < kN; e += 2) turn(p.x[e], p.x[e + 1], cs[(i * kN + e) / 2]);
          v = p.get();
        }
        *reinterpret_cast<uint4 *>(to + i * 16) = v;
      }
    } else {
      const int half = r.pairs / kN;
      for (int i = lane; i < pieces - half; i += lanes) {
        if (i < half) {
          Piece<E> a, b;
          a.load(from + i * 16);
          b.load(from + (i + half) * 16);
#pragma unroll
          for (int e = 0; e < kN; ++e) turn(a.x[e], b.x[e], cs[i * kN + e]);
          *reinterpret_cast<uint4 *>(to + i * 16) = a.get();
          *reinterpret_cast<uint4 *>(to + (i + half) * 16) = b.get();
        } else if (from != to) {
          *reinterpret_cast<uint4 *>(to + (i + half) * 16) =
              *reinterpret_cast<const uint4 *>(from + (i + half) * 16);
        }
      }
    }
  } else {
    const T *x = reinterpret_cast<const T *>(from);
    T *y = reinterpret_cast<T *>(to);
    for (int i = lane; i < D - r.pairs; i += lanes) {
      if (i < r.pairs) {
        const int i0 = r.interleaved ? 2 * i : i, i1 = r.interleaved ? 2 * i + 1 : i + r.pairs;
        float a = E::to(x[i0]), b = E::to(x[i1]);
        turn(a, b, cs[i]);
        y[i0] = E::from(a);
        y[i1] = E::from(b);
      } else if (from != to) {
        y[i + r.pairs] = x[i + r.pairs];
      }
    }
  }
}

// Eight values of a row from element 8 * i on, rotated.
template <class E, bool kVector>
__device__ __forceinline__ void rotated8(const char *row, int i, const Rotation &r, const float2 *cs,
                                         float (&x)[8]) {
  using T = typename E::T;
  constexpr int kN = Piece<E>::kN;
  auto load8 = [&](int e0, float (&y)[8]) {
#pragma unroll
    for (int e = 0; e < 8; e += kN) {
      Piece<E> p;
      p.load(row + (e0 + e) * sizeof(T));
#pragma unroll
      for (int j = 0; j < kN; ++j) y[e + j] = p.x[j];
    }
  };
  load8(8 * i, x);
  if (8 * i >= 2 * r.pairs) return;
  if (kVector && r.interleaved) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) turn(x[e], x[e + 1], cs[4 * i + e / 2]);
  } else if (kVector) {
    const bool second = 8 * i >= r.pairs;
    const int pair0 = second ? 8 * i - r.pairs : 8 * i;
    float y[8];
    load8(second ? pair0 : pair0 + r.pairs, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float a = second ? y[e] : x[e], b = second ? x[e] : y[e];
      turn(a, b, cs[pair0 + e]);
      x[e] = second ? b : a;
    }
  } else {
    const T *t = reinterpret_cast<const T *>(row);
    for (int e = 0; e < 8; ++e) {
      const int at = 8 * i + e;
      if (at >= 2 * r.pairs) break;
      const bool second = r.interleaved ? at & 1 : at >= r.pairs;
      const int pair = r.interleaved ? at / 2 : (second ? at - r.pairs : at);
      float a = E::to(t[r.interleaved ? 2 * pair : pair]);
      float b = E::to(t[r.interleaved ? 2 * pair + 1 : pair + r.pairs]);
      turn(a, b, cs[pair]);
      x[e] = second ? b : a;
    }
  }
  // the rows are made of keys in the type that they come in
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = E::to(E::from(x[e]));
}

// One row as a 4-bit row, by the D / 8 neighbouring lanes of which this is the
// lane-th (whole warps call it); x: its values.
__device__ __forceinline__ void write_q4(char *to, int D, int lane, float (&x)[8], bool there) {
  const int words = D / 8, per = words / kQ4Groups;  // lanes of a group: 2, 4 (D 64, 128)
  float lo = INFINITY, hi = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    bad |= !isfinite(x[e]);
    x[e] = fminf(fmaxf(x[e], -kQ4Limit), kQ4Limit);
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
  }
  for (int o = 1; o < per; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
    bad |= __shfl_xor_sync(0xFFFFFFFFu, static_cast<int>(bad), o) != 0;
  }
  const Q4Scale q = q4_scale(lo, hi, bad);
  const uint32_t word = q4_word(q, x);
  if (!there) return;
  *reinterpret_cast<uint32_t *>(to + lane * 4) = word;
  if (lane % per == 0) *reinterpret_cast<uint32_t *>(to + D / 2 + lane / per * 4) = q.bits;
}

__device__ __forceinline__ char *at_row(const TokenRows &t, long long layer, int b, int n) {
  return t.data + layer * t.layer + b * t.seq + n * t.token;
}

// A token of a batch: what find_token looks up once.
struct Token {
  int b, n;          // n < 0: none, or behind the sequence's new tokens
  long long k, v;    // byte offsets of its slot's first head; -1: not written
  long long place;   // position
};

// ---------------------------------------------------------------------------
// queries rotated, keys rotated and written, values written
// ---------------------------------------------------------------------------

struct AppendArgs {
  KvSeqs S;
  KvCache C;
  RotaryRows R;
  Rotation rotation;
  int D, batch, row_lanes;  // tokens of a CTA; threads of a row
};

template <class E, bool kFour, bool kVector>
__global__ void __launch_bounds__(kRotThreads) append_rotary_kernel(const __grid_constant__ AppendArgs a) {
  extern __shared__ float2 cs[];  // batch x pairs
  __shared__ Token tokens[kRotThreads];
  const int tid = threadIdx.x, layer = blockIdx.y;
  const long long total = static_cast<long long>(a.S.B) * a.S.N, t0 = static_cast<long long>(blockIdx.x) * a.batch;
  const int count = static_cast<int>(min(static_cast<long long>(a.batch), total - t0));
  if (tid < count) {
    Token t;
    t.b = static_cast<int>((t0 + tid) / a.S.N);
    t.n = static_cast<int>(t0 + tid - static_cast<long long>(t.b) * a.S.N);
    t.k = t.v = -1;
    const int ctx = __ldg(a.S.ctx + t.b), m = seq_new(a.S, t.b);
    int behind = t.n;
    if (a.R.position)
      behind = min(max(__ldg(a.R.position + t.b * a.R.position_seq + t.n), 0), a.S.N - 1);
    t.place = static_cast<long long>(ctx) + behind;
    if (t.n >= m) {
      t.n = -1;
    } else if (seq_fits(a.S, a.C, ctx, m)) {
      const int at = ctx + t.n, index = at / a.C.page_size, page = page_at(a.S, t.b, index);
      if (page_ok(a.C, page)) {
        const int in_page = at - index * a.C.page_size;
        t.k = layer * a.C.k_layer + page * a.C.k_page + in_page * a.C.k_token;
        t.v = layer * a.C.v_layer + page * a.C.v_page + in_page * a.C.v_token;
      }
    }
    tokens[tid] = t;
  }
  __syncthreads();
  if (a.rotation.pairs > 0)
    find_angles(a.rotation, count, [&](int i) { return tokens[i].place; }, cs);
  const int lane = tid % a.row_lanes, group = tid / a.row_lanes, groups = kRotThreads / a.row_lanes;
  if (a.R.q.data) {
    const int heads = a.R.q_heads;
    for (int i = group; i < count * heads; i += groups) {
      const int token = i / heads, h = i - token * heads;
      const Token &t = tokens[token];
      if (t.n < 0) continue;
      rotate_row<E, kVector>(at_row(a.R.q, layer, t.b, t.n) + h * a.R.q.head,
                             at_row(a.R.out_q, layer, t.b, t.n) + h * a.R.out_q.head, a.D, a.rotation,
                             cs + token * a.rotation.pairs, lane, a.row_lanes);
    }
  }
  const int heads = a.C.heads, rows = 2 * heads;
  if constexpr (!kFour) {
    for (int i = group; i < count * rows; i += groups) {
      const int token = i / rows, r = i - token * rows;
      const Token &t = tokens[token];
      if (t.n < 0) continue;
      if (r < heads) {
        if (t.k >= 0)
          rotate_row<E, kVector>(at_row(a.R.k, layer, t.b, t.n) + r * a.R.k.head,
                                 a.C.k + t.k + r * a.C.k_head, a.D, a.rotation,
                                 cs + token * a.rotation.pairs, lane, a.row_lanes);
      } else if (t.v >= 0) {
        const char *from = at_row(a.R.v, layer, t.b, t.n) + (r - heads) * a.R.v.head;
        char *to = a.C.v + t.v + (r - heads) * a.C.v_head;
        for (int p = lane; p < a.C.row_bytes / 16; p += a.row_lanes)
          *reinterpret_cast<uint4 *>(to + p * 16) = *reinterpret_cast<const uint4 *>(from + p * 16);
      }
    }
  } else {
    const int words = a.D / 8, word = tid % words, each = kRotThreads / words;
    // whole warps stay together for the groups' shuffles
    for (int i0 = 0; i0 < count * rows; i0 += each) {
      const int i = i0 + tid / words, token = min(i / rows, count - 1), r = i % rows;
      const Token &t = tokens[token];
      const bool is_k = r < heads;
      const bool there = i < count * rows && t.n >= 0 && (is_k ? t.k : t.v) >= 0;
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (there) {
        if (is_k) {
          rotated8<E, kVector>(at_row(a.R.k, layer, t.b, t.n) + r * a.R.k.head, word, a.rotation,
                               cs + token * a.rotation.pairs, x);
        } else {
          Rotation none = {};
          rotated8<E, true>(at_row(a.R.v, layer, t.b, t.n) + (r - heads) * a.R.v.head, word, none, cs, x);
        }
      }
      write_q4(is_k ? a.C.k + t.k + r * a.C.k_head : a.C.v + t.v + (r - heads) * a.C.v_head, a.D, word,
               x, there);
    }
  }
}

// ---------------------------------------------------------------------------
// rows rotated
// ---------------------------------------------------------------------------

struct RotateArgs {
  TokenRows x, out;
  const int32_t *position;
  long long position_seq;
  Rotation rotation;
  int B, N, heads, D, batch, row_lanes;
};

template <class E, bool kVector>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotateArgs a) {
  extern __shared__ float2 cs[];
  __shared__ long long from[kRotThreads], to[kRotThreads];
  const int tid = threadIdx.x;
  const long long total = static_cast<long long>(a.B) * a.N, t0 = static_cast<long long>(blockIdx.x) * a.batch;
  const int count = static_cast<int>(min(static_cast<long long>(a.batch), total - t0));
  if (tid < count) {
    const int b = static_cast<int>((t0 + tid) / a.N), n = static_cast<int>(t0 + tid - static_cast<long long>(b) * a.N);
    from[tid] = b * a.x.seq + n * a.x.token;
    to[tid] = b * a.out.seq + n * a.out.token;
  }
  // behind the barrier of find_angles
  find_angles(a.rotation, count, [&](int i) {
    const long long t = t0 + i, b = t / a.N;
    return static_cast<long long>(__ldg(a.position + b * a.position_seq + (t - b * a.N)));
  }, cs);
  const int lane = tid % a.row_lanes, group = tid / a.row_lanes, groups = kRotThreads / a.row_lanes;
  for (int i = group; i < count * a.heads; i += groups) {
    const int token = i / a.heads, h = i - token * a.heads;
    rotate_row<E, kVector>(a.x.data + from[token] + h * a.x.head, a.out.data + to[token] + h * a.out.head,
                           a.D, a.rotation, cs + token * a.rotation.pairs, lane, a.row_lanes);
  }
}

// ---------------------------------------------------------------------------
// rows read back
// ---------------------------------------------------------------------------

struct ReadArgs {
  KvSeqs S;
  KvCache C;
  TokenRows k, v;
  int D;
};

// A warp takes a token: its slot once, then its keys and values in a layer.
template <class E, bool kFour>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs a) {
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31, layer = blockIdx.y;
  if (t >= a.S.B * a.S.N) return;
  const int b = t / a.S.N, n = t - b * a.S.N;
  const int start = __ldg(a.S.ctx + b), m = seq_new(a.S, b);
  const char *k = nullptr, *v = nullptr;
  if (n < m && seq_fits(a.S, a.C, start, m)) {
    const int at = start + n, index = at / a.C.page_size, page = page_at(a.S, b, index);
    if (page_ok(a.C, page)) {
      const int in_page = at - index * a.C.page_size;
      k = a.C.k + layer * a.C.k_layer + page * a.C.k_page + in_page * a.C.k_token;
      v = a.C.v + layer * a.C.v_layer + page * a.C.v_page + in_page * a.C.v_token;
    }
  }
  char *k_out = at_row(a.k, layer, b, n), *v_out = at_row(a.v, layer, b, n);
  const int heads = a.C.heads;
  if constexpr (!kFour) {
    const int per_row = a.C.row_bytes / 16, rows = 2 * heads;
    for (int i = lane; i < rows * per_row; i += 32) {
      const int r = i / per_row, c = (i - r * per_row) * 16;
      const bool is_k = r < heads;
      const int h = is_k ? r : r - heads;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (k) x = *reinterpret_cast<const uint4 *>((is_k ? k + h * a.C.k_head : v + h * a.C.v_head) + c);
      *reinterpret_cast<uint4 *>((is_k ? k_out + h * a.k.head : v_out + h * a.v.head) + c) = x;
    }
  } else {
    const int words = a.D / 8, per = words / kQ4Groups;
    for (int i = lane; i < 2 * heads * words; i += 32) {
      const int r = i / words, w = i - r * words;
      const bool is_k = r < heads;
      const int h = is_k ? r : r - heads;
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (k) {
        const char *row = is_k ? k + h * a.C.k_head : v + h * a.C.v_head;
        q4_codes(*reinterpret_cast<const uint32_t *>(row + w * 4), x);
        const float2 s = q4_pair(*reinterpret_cast<const uint32_t *>(row + a.D / 2 + w / per * 4));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(s.x, x[e], s.y);
      }
      char *to = (is_k ? k_out + h * a.k.head : v_out + h * a.v.head) + w * 8 * sizeof(typename E::T);
      constexpr int kN = Piece<E>::kN;
#pragma unroll
      for (int e = 0; e < 8; e += kN) {
        Piece<E> p;
#pragma unroll
        for (int j = 0; j < kN; ++j) p.x[j] = x[e + j];
        *reinterpret_cast<uint4 *>(to + e * sizeof(typename E::T)) = p.get();
      }
    }
  }
}

// Whether pairs fall on whole pieces of n values.
bool whole_pieces(const Rotation &r, int n) { return (r.interleaved ? 2 * r.pairs : r.pairs) % n == 0; }

// Threads of a row: as many as it has pieces (of a pair's two halves one), rounded up
// to a power of two.
int lanes_of(int D, int n, const Rotation &r, bool vector) {
  const int items = vector ? D / n - (r.interleaved ? 0 : r.pairs / n) : D - r.pairs;
  int lanes = 1;
  while (lanes < items && lanes < kRotThreads) lanes <<= 1;
  return lanes;
}

// Tokens of a CTA: as many as threads find angles for at once, fewer where that
// leaves SMs without work.
int batch_of(long long tokens, int layers, int pairs) {
  const int most = pairs > 0 ? std::max(1, kRotThreads / pairs) : 4;
  const long long spread = tokens * layers / (4 * 152);
  return static_cast<int>(std::max<long long>(1, std::min<long long>(std::min(most, 16), spread)));
}

template <class F>
cudaError_t by_type(int dtype, F f) {
  if (dtype == SPEC_F32) return f(F32());
  if (dtype == SPEC_BF16) return f(Bf16());
  return f(F16());
}

}  // namespace

cudaError_t launch_append_rotary(const KvSeqs &S, const KvCache &C, const RotaryRows &R, int D,
                                 int dtype, bool four, const Rotation &rotation, uint32_t *flags,
                                 cudaStream_t stream) {
  if (flags) {
    const cudaError_t e = launch_kv_flags(S, C, true, 0, 0, flags, stream);
    if (e != cudaSuccess) return e;
  }
  const long long tokens = static_cast<long long>(S.B) * S.N;
  if (tokens == 0) return cudaSuccess;
  return by_type(dtype, [&](auto type) {
    using E = decltype(type);
    constexpr int kN = Piece<E>::kN;
    const bool vector = whole_pieces(rotation, kN) && (!four || whole_pieces(rotation, 8));
    AppendArgs a = {S, C, R, rotation, D, batch_of(tokens, C.layers, rotation.pairs),
                    lanes_of(D, kN, rotation, vector)};
    const dim3 grid(static_cast<unsigned>((tokens + a.batch - 1) / a.batch), C.layers);
    const size_t smem = static_cast<size_t>(a.batch) * rotation.pairs * sizeof(float2);
    if (four) {
      if (vector) {
        append_rotary_kernel<E, true, true><<<grid, kRotThreads, smem, stream>>>(a);
      } else {
        append_rotary_kernel<E, true, false><<<grid, kRotThreads, smem, stream>>>(a);
      }
    } else if (vector) {
      append_rotary_kernel<E, false, true><<<grid, kRotThreads, smem, stream>>>(a);
    } else {
      append_rotary_kernel<E, false, false><<<grid, kRotThreads, smem, stream>>>(a);
    }
    return cudaGetLastError();
  });
}

cudaError_t launch_rotary(const TokenRows &x, const TokenRows &out, int dtype, int B, int N, int heads,
                          int D, const int32_t *position, long long position_seq,
                          const Rotation &rotation, cudaStream_t stream) {
  const long long tokens = static_cast<long long>(B) * N;
  if (tokens == 0 || heads == 0) return cudaSuccess;
  return by_type(dtype, [&](auto type) {
    using E = decltype(type);
    constexpr int kN = Piece<E>::kN;
    auto on_pieces = [&](const TokenRows &t) {
      return ((reinterpret_cast<uintptr_t>(t.data) | (B > 1 ? t.seq : 0) | (N > 1 ? t.token : 0) |
               (heads > 1 ? t.head : 0)) & 15) == 0;
    };
    const bool vector = whole_pieces(rotation, kN) && D % kN == 0 && on_pieces(x) && on_pieces(out);
    const RotateArgs a = {x, out, position, position_seq, rotation, B, N, heads, D,
                          batch_of(tokens, 1, rotation.pairs), lanes_of(D, kN, rotation, vector)};
    const unsigned grid = static_cast<unsigned>((tokens + a.batch - 1) / a.batch);
    const size_t smem = static_cast<size_t>(a.batch) * rotation.pairs * sizeof(float2);
    if (vector) {
      rotary_kernel<E, true><<<grid, kRotThreads, smem, stream>>>(a);
    } else {
      rotary_kernel<E, false><<<grid, kRotThreads, smem, stream>>>(a);
    }
    return cudaGetLastError();
  });
}

cudaError_t launch_read(const KvSeqs &S, const KvCache &C, const TokenRows &k, const TokenRows &v, int D,
                        int dtype, bool four, uint32_t *flags, cudaStream_t stream) {
  if (flags) {
    const cudaError_t e = launch_kv_flags(S, C, true, 0, 0, flags, stream);
    if (e != cudaSuccess) return e;
  }
  const int tokens = S.B * S.N;
  if (tokens == 0) return cudaSuccess;
  return by_type(dtype, [&](auto type) {
    using E = decltype(type);
    const ReadArgs a = {S, C, k, v, D};
    const dim3 grid((tokens + kWarps - 1) / kWarps, C.layers);
    if (four) {
      read_kernel<E, true><<<grid, kThreads, 0, stream>>>(a);
    } else {
      read_kernel<E, false><<<grid, kThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
  });
}

}  // namespace sv
