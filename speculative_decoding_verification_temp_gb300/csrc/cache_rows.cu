// New tokens' rows on their way into the paged cache and out of it: queries and
// keys rotated by their positions, keys and values written to their pages as they
// are or as 4-bit rows (q4.cuh), and read back.
//
// Rotation: a pair (a, b) of a head's values becomes (a cos t - b sin t, a sin t +
// b cos t), t = position * frequency.  Far positions times frequencies lose their
// angle in float32, and float64 is slow here, so a frequency becomes the fraction of
// a turn per token in 64-bit fixed point once per thread; an integer product that
// wraps is then the angle itself, off by 2^-64 turns per token of position, and
// sine and cosine see a float32 in [-1/2, 1/2] turns.  A CTA takes a batch of tokens
// (kRotThreads / pairs at most): one thread per (token, pair) finds the angle, and all
// of the tokens' heads use it from shared memory.
//
// Rows are read once and written once, in 16-byte pieces, a thread holding both pieces of
// its pairs, so that queries may be rotated in place.  Two rows a thread in flight (one 64 us,
// four 61) on six thread blocks an SM (three 61, eight 64): 16384 tokens' 40 heads of 128,
// bf16, 55 us, 0.90 of the copy rate.  Appends find their slots through three loads one behind
// another before they read: five prompts of up to 4001 tokens, 32/8 heads of 128, f16, 60 us,
// 0.61 of it.  4-bit rows are bound by instructions, a minimum, a maximum and a code per value:
// 8192 tokens, 32/8 heads of 64, 28 us with the queries' rotation.
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

// A thread's frequency as turns per token, in units of 2^-64 turns, wrapped.  1 / (2 pi) has
// 128 bits behind the point, times a mantissa of 53: good to that unit for frequencies up to
// 2^53, and by integers faster than the same by float64 (16384 tokens' 40 heads 59 us for
// 57).  Larger ones, by sums of two float64: good to 2^-106 of themselves.
__device__ __forceinline__ unsigned long long turn_of(double frequency) {
  constexpr unsigned long long kHigh = 0x28BE60DB9391054Aull, kLow = 0x7F09D5F47D4D3770ull;
  const long long bits = __double_as_longlong(frequency);
  const int exponent = static_cast<int>(bits >> 52 & 2047) - 1023;
  unsigned long long turn;
  if (exponent <= 52) {
    const unsigned long long mantissa = (bits & ((1ll << 52) - 1)) | 1ll << 52;
    const unsigned long long carry = __umul64hi(mantissa, kLow), part = mantissa * kHigh, low = part + carry;
    const unsigned long long high = __umul64hi(mantissa, kHigh) + (low < part ? 1 : 0);
    const int down = 52 - exponent;
    turn = down >= 64 ? (down < 128 ? high >> (down - 64) : 0) : (low >> down | (down ? high << (64 - down) : 0));
  } else {
    constexpr double kUnits = 18446744073709551616.0;
    const double x = fabs(frequency), a = x * 0.15915494309189535, b = fma(x, -9.839338337591243e-18, fma(x, 0.15915494309189535, -a));
    turn = static_cast<unsigned long long>(__double2ll_rn((a - rint(a)) * kUnits)) +
           static_cast<unsigned long long>(__double2ll_rn((b - rint(b)) * kUnits));
  }
  return bits < 0 ? 0 - turn : turn;
}

// Where a pair's angle is: neighbouring lanes take neighbouring pieces of kEach pairs, and
// of a piece one pair at a time, so that the first pairs of all pieces come first, then the
// second ones (pairs in order, of which four lanes meet a bank, and a row at a time: prompts'
// rows 84 us, 61 so with four rows at once).
template <int kEach>
__device__ __forceinline__ int angle_at(int pairs, int pair) {
  return pair % kEach * (pairs / kEach) + pair / kEach;
}

// cos and sin of every (token of the batch, pair), by the whole CTA; place(i): the
// position of token i of the batch; each: of angle_at.  Ends with a barrier.
template <class Place>
__device__ __forceinline__ void find_angles(const Rotation &r, int tokens, Place place, float2 *cs, int each) {
  // pairs <= kRotThreads: a thread keeps its pair
  const int per = kRotThreads / r.pairs, pair = threadIdx.x % r.pairs;
  const int first = threadIdx.x / r.pairs;
  if (first < per && first < tokens) {
    const double f = __ldg(r.frequency + pair);
    const int to = pair % each * (r.pairs / each) + pair / each;
    const unsigned long long turn = turn_of(f);
    for (int i = first; i < tokens; i += per) {
      const long long at = place(i);
      // two's complement: the fraction nearest to zero
      const long long fraction = static_cast<long long>(turn * static_cast<unsigned long long>(at));
      float s, c;
      // fraction * 2^-64 turns are fraction * 2^-63 half turns
      sincospif(static_cast<float>(fraction) * 1.0842021724855044e-19f, &s, &c);
      if (!isfinite(f)) s = c = __int_as_float(0x7FC00000);
      cs[i * r.pairs + to] = make_float2(c * r.amplitude, (r.inverse ? -s : s) * r.amplitude);
    }
  }
  __syncthreads();
}

__device__ __forceinline__ void turn(float &a, float &b, float2 cs) {
  const float x = fmaf(a, cs.x, -(b * cs.y));
  b = fmaf(a, cs.y, b * cs.x);
  a = x;
}

// Pairs of a piece (angle_at); pairs that do not fall on whole pieces stay in order.
template <class E, bool kVector>
__device__ __forceinline__ int each_of(const Rotation &r) {
  constexpr int kN = Piece<E>::kN;
  return !kVector || r.pairs == 0 ? 1 : (r.interleaved ? kN / 2 : kN);
}

// A row to rotate: angles NULL: there is none.
struct RowJob {
  const char *from;
  char *to;
  const float2 *angles;
};

constexpr int kAtOnce = 2, kFourAtOnce = 1;

// Walks the (token, head) rows of a batch, every groups-th of them.
struct RowWalk {
  int token, h, heads, step_token, step_h;
  __device__ __forceinline__ RowWalk(int heads, int group, int groups)
      : token(group / heads), h(group - token * heads), heads(heads), step_token(groups / heads),
        step_h(groups - step_token * heads) {}
  __device__ __forceinline__ void next() {
    token += step_token;
    h += step_h;
    if (h >= heads) {
      h -= heads;
      ++token;
    }
  }
};

// The heads' rows of `count` tokens rotated, the first of them this thread's group's, then
// every groups-th, by the `lanes` threads of which this is the lane-th.  kVector: the
// pairs' halves begin at 16-byte pieces; of kAtOnce rows all pieces are asked for before
// the first is written.
template <class E, bool kVector, class Job>
__device__ __forceinline__ void rotate_rows(int count, int heads, int group, int groups, int D, const Rotation &r,
                                            int lane, int lanes, Job job) {
  using T = typename E::T;
  constexpr int kN = Piece<E>::kN;
  if constexpr (kVector) {
    // a lane has a piece, or one of each half
    const int pieces = D / kN, half = r.interleaved ? 0 : r.pairs / kN;
    const int turned = r.interleaved ? 2 * r.pairs / kN : half;
    for (int i = lane; i < pieces - half; i += lanes) {
      const bool turns = i < turned, two = turns && !r.interleaved;
      const int first = turns ? i : i + half;
      for (RowWalk w(heads, group, groups); w.token < count;) {
        uint4 a[kAtOnce], b[kAtOnce];
        RowJob jobs[kAtOnce];
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x, w.next()) {
          jobs[x].angles = nullptr;
          if (w.token >= count) continue;
          jobs[x] = job(w.token, w.h);
          if (!jobs[x].angles) continue;
          a[x] = *reinterpret_cast<const uint4 *>(jobs[x].from + first * 16);
          if (two) b[x] = *reinterpret_cast<const uint4 *>(jobs[x].from + (i + half) * 16);
        }
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
          if (!jobs[x].angles) continue;
          if (two) {
            Piece<E> y, z;
            y.set(a[x]);
            z.set(b[x]);
#pragma unroll
            for (int e = 0; e < kN; ++e) turn(y.x[e], z.x[e], jobs[x].angles[e * half + i]);
            a[x] = y.get();
            *reinterpret_cast<uint4 *>(jobs[x].to + (i + half) * 16) = z.get();
          } else if (turns) {
            Piece<E> y;
            y.set(a[x]);
#pragma unroll
            for (int e = 0; e < kN; e += 2) turn(y.x[e], y.x[e + 1], jobs[x].angles[e / 2 * turned + i]);
            a[x] = y.get();
          }
          *reinterpret_cast<uint4 *>(jobs[x].to + first * 16) = a[x];
        }
      }
    }
  } else {
    for (RowWalk w(heads, group, groups); w.token < count; w.next()) {
      const RowJob j = job(w.token, w.h);
      if (!j.angles) continue;
      const T *x = reinterpret_cast<const T *>(j.from);
      T *y = reinterpret_cast<T *>(j.to);
      for (int i = lane; i < D - r.pairs; i += lanes) {
        if (i < r.pairs) {
          const int i0 = r.interleaved ? 2 * i : i, i1 = r.interleaved ? 2 * i + 1 : i + r.pairs;
          float a = E::to(x[i0]), b = E::to(x[i1]);
          turn(a, b, j.angles[i]);
          y[i0] = E::from(a);
          y[i1] = E::from(b);
        } else if (j.from != j.to) {
          y[i + r.pairs] = x[i + r.pairs];
        }
      }
    }
  }
}

// Eight values of a row.
template <class E>
struct Eight {
  static constexpr int kN = Piece<E>::kN;
  uint4 v[8 / kN];
  __device__ __forceinline__ void load(const char *row, int e0) {
#pragma unroll
    for (int i = 0; i < 8 / kN; ++i)
      v[i] = *reinterpret_cast<const uint4 *>(row + e0 * sizeof(typename E::T) + i * 16);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8 / kN; ++i) {
      Piece<E> p;
      p.set(v[i]);
#pragma unroll
      for (int j = 0; j < kN; ++j) x[i * kN + j] = p.x[j];
    }
  }
};

// A lane's part of a row that becomes a 4-bit one: eight values from element 8 * i on, and
// with kVector the other values of their pairs.
template <class E, bool kVector>
struct RowPart {
  Eight<E> own, other;
  // 0: as they are, 1: neighbours are pairs, 2, 3: first, second values of pairs
  __device__ __forceinline__ static int how(int i, const Rotation &r) {
    return 8 * i >= 2 * r.pairs ? 0 : (r.interleaved ? 1 : (8 * i >= r.pairs ? 3 : 2));
  }
  __device__ __forceinline__ void load(const char *row, int i, const Rotation &r) {
    own.load(row, 8 * i);
    if (kVector && how(i, r) >= 2) other.load(row, how(i, r) == 3 ? 8 * i - r.pairs : 8 * i + r.pairs);
  }
  __device__ __forceinline__ void rotated(const char *row, int i, const Rotation &r, const float2 *cs,
                                          float (&x)[8]) const {
    using T = typename E::T;
    constexpr int kN = Piece<E>::kN;
    own.get(x);
    const int kind = how(i, r);
    if (kind == 0) return;
    if (kVector && kind == 1) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) turn(x[e], x[e + 1], cs[angle_at<kN / 2>(r.pairs, 4 * i + e / 2)]);
    } else if (kVector) {
      const bool second = kind == 3;
      const int pair0 = second ? 8 * i - r.pairs : 8 * i;
      float y[8];
      other.get(y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float2 t = cs[angle_at<kN>(r.pairs, pair0 + e)];
        // b cos + a sin, a cos - b sin
        if (!second) t.y = -t.y;
        x[e] = second ? fmaf(y[e], t.y, x[e] * t.x) : fmaf(x[e], t.x, y[e] * t.y);
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
};

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

constexpr int kMaxBatch = 16;

// A token of a batch: byte offsets of its first heads' rows.
struct Token {
  long long q, out_q, k, v, to_k, to_v;  // to_k < 0: not written
  long long place;                       // position
  bool there;                            // not behind the sequence's new tokens
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
__global__ void __launch_bounds__(kRotThreads, 5) append_rotary_kernel(const __grid_constant__ AppendArgs a) {
  extern __shared__ float2 cs[];  // batch x pairs
  __shared__ Token tokens[kMaxBatch];
  const int tid = threadIdx.x, layer = blockIdx.y;
  const long long total = static_cast<long long>(a.S.B) * a.S.N, t0 = static_cast<long long>(blockIdx.x) * a.batch;
  const int count = static_cast<int>(min(static_cast<long long>(a.batch), total - t0));
  if (tid < count) {
    Token t;
    const int b = static_cast<int>((t0 + tid) / a.S.N);
    const int n = static_cast<int>(t0 + tid - static_cast<long long>(b) * a.S.N);
    auto offset = [&](const TokenRows &x) { return layer * x.layer + b * x.seq + n * x.token; };
    t.q = offset(a.R.q);
    t.out_q = offset(a.R.out_q);
    t.k = offset(a.R.k);
    t.v = offset(a.R.v);
    t.to_k = t.to_v = -1;
    const int ctx = __ldg(a.S.ctx + b), m = seq_new(a.S, b);
    int behind = n;
    if (a.R.position) behind = min(max(__ldg(a.R.position + b * a.R.position_seq + n), 0), a.S.N - 1);
    t.place = static_cast<long long>(ctx) + behind;
    t.there = n < m;
    if (t.there && seq_fits(a.S, a.C, ctx, m)) {
      const int at = ctx + n, index = at / a.C.page_size, page = page_at(a.S, b, index);
      if (page_ok(a.C, page)) {
        const int in_page = at - index * a.C.page_size;
        t.to_k = layer * a.C.k_layer + page * a.C.k_page + in_page * a.C.k_token;
        t.to_v = layer * a.C.v_layer + page * a.C.v_page + in_page * a.C.v_token;
      }
    }
    tokens[tid] = t;
  }
  __syncthreads();
  if (a.rotation.pairs > 0)
    find_angles(a.rotation, count, [&](int i) { return tokens[i].place; }, cs, each_of<E, kVector>(a.rotation));
  const int lane = tid % a.row_lanes, group = tid / a.row_lanes, groups = kRotThreads / a.row_lanes;
  if (a.R.q.data)
    rotate_rows<E, kVector>(
        count, a.R.q_heads, group, groups, a.D, a.rotation, lane, a.row_lanes, [&](int token, int h) {
          const Token &t = tokens[token];
          return RowJob{a.R.q.data + t.q + h * a.R.q.head, a.R.out_q.data + t.out_q + h * a.R.out_q.head,
                        t.there ? cs + token * a.rotation.pairs : nullptr};
        });
  const int heads = a.C.heads, rows = 2 * heads;
  if constexpr (!kFour) {
    rotate_rows<E, kVector>(
        count, heads, group, groups, a.D, a.rotation, lane, a.row_lanes, [&](int token, int h) {
          const Token &t = tokens[token];
          return RowJob{a.R.k.data + t.k + h * a.R.k.head, a.C.k + t.to_k + h * a.C.k_head,
                        t.to_k >= 0 ? cs + token * a.rotation.pairs : nullptr};
        });
    for (int piece = lane; piece < a.C.row_bytes / 16; piece += a.row_lanes)
      for (RowWalk w(heads, group, groups); w.token < count;) {
        uint4 x[kAtOnce];
        char *to[kAtOnce];
#pragma unroll
        for (int y = 0; y < kAtOnce; ++y, w.next()) {
          to[y] = nullptr;
          if (w.token >= count) continue;
          const Token &t = tokens[w.token];
          if (t.to_k < 0) continue;
          to[y] = a.C.v + t.to_v + w.h * a.C.v_head + piece * 16;
          x[y] = *reinterpret_cast<const uint4 *>(a.R.v.data + t.v + w.h * a.R.v.head + piece * 16);
        }
#pragma unroll
        for (int y = 0; y < kAtOnce; ++y)
          if (to[y]) *reinterpret_cast<uint4 *>(to[y]) = x[y];
      }
  } else {
    const int words = a.D / 8, word = tid % words, each = kRotThreads / words;
    const Rotation none = {};
    // whole warps stay together for the groups' shuffles
    RowWalk w(rows, tid / words, each);
    for (int i0 = 0; i0 < count * rows; i0 += kFourAtOnce * each) {
      RowPart<E, kVector> part[kFourAtOnce];
      const char *from[kFourAtOnce];
      char *to[kFourAtOnce];
      int of[kFourAtOnce];  // token; negative: of a value
#pragma unroll
      for (int y = 0; y < kFourAtOnce; ++y, w.next()) {
        from[y] = nullptr;
        if (w.token >= count) continue;
        const Token &t = tokens[w.token];
        if (t.to_k < 0) continue;
        const bool is_k = w.h < heads;
        from[y] = is_k ? a.R.k.data + t.k + w.h * a.R.k.head : a.R.v.data + t.v + (w.h - heads) * a.R.v.head;
        to[y] = is_k ? a.C.k + t.to_k + w.h * a.C.k_head : a.C.v + t.to_v + (w.h - heads) * a.C.v_head;
        of[y] = is_k ? w.token : -1;
        part[y].load(from[y], word, is_k ? a.rotation : none);
      }
#pragma unroll
      for (int y = 0; y < kFourAtOnce; ++y) {
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (from[y]) {
          if (of[y] < 0) {
            part[y].own.get(x);
          } else {
            part[y].rotated(from[y], word, a.rotation, cs + of[y] * a.rotation.pairs, x);
          }
        }
        write_q4(to[y], a.D, word, x, from[y] != nullptr);
      }
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
__global__ void __launch_bounds__(kRotThreads, 6) rotary_kernel(const __grid_constant__ RotateArgs a) {
  extern __shared__ float2 cs[];
  __shared__ long long from[kMaxBatch], to[kMaxBatch];
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
  }, cs, each_of<E, kVector>(a.rotation));
  const int lane = tid % a.row_lanes, group = tid / a.row_lanes, groups = kRotThreads / a.row_lanes;
  rotate_rows<E, kVector>(
      count, a.heads, group, groups, a.D, a.rotation, lane, a.row_lanes, [&](int token, int h) {
        return RowJob{a.x.data + from[token] + h * a.x.head, a.out.data + to[token] + h * a.out.head,
                      cs + token * a.rotation.pairs};
      });
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
  return static_cast<int>(std::max<long long>(1, std::min<long long>(std::min(most, kMaxBatch), spread)));
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
