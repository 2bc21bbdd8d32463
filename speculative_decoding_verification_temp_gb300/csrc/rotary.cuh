// What the rotation's kernels take.
#pragma once

#include "kv_cache.cuh"

namespace sv {

constexpr int kMaxPairs = 256;  // of a head

// Rotation by position: pair i turns by position * frequency[i] radians.
struct Rotation {
  const double *frequency;  // NULL: none
  int pairs;
  bool interleaved, inverse;
  float amplitude;
};

// Rows of tokens; strides in bytes.
struct TokenRows {
  char *data;
  long long layer, seq, token, head;
};

// New tokens' rows: queries (q.data NULL: none), keys and values.
struct RotaryRows {
  TokenRows q, out_q, k, v;
  int q_heads;
  const int32_t *position;  // of the new tokens behind the context; NULL: 0, 1, ...
  long long position_seq;
};

// dtype: of the rows.  four: the cache's rows are 4-bit ones.
cudaError_t launch_append_rotary(const KvSeqs &S, const KvCache &C, const RotaryRows &R, int D,
                                 int dtype, bool four, const Rotation &rotation, uint32_t *flags,
                                 cudaStream_t stream);
// heads of [B, N] tokens at position[b * position_seq + n]; x and out are the same rows or
// do not overlap.
cudaError_t launch_rotary(const TokenRows &x, const TokenRows &out, int dtype, int B, int N, int heads,
                          int D, const int32_t *position, long long position_seq,
                          const Rotation &rotation, cudaStream_t stream);
// Tokens start[b] + n, n < num[b], of each sequence as rows; zeros for the others.
cudaError_t launch_read(const KvSeqs &S, const KvCache &C, const TokenRows &k, const TokenRows &v, int D,
                        int dtype, bool four, uint32_t *flags, cudaStream_t stream);

}  // namespace sv
