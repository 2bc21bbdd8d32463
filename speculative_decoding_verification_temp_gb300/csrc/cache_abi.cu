// C ABI of the paged key-value cache operators: argument checks and the
// kernels' views of the caller's arrays.  The operations are documented in
// include/specverify.h.
#include <climits>
#include <cmath>
#include <cstdint>

#include "paged_attention.cuh"

namespace sv {
cudaError_t launch_append(const KvSeqs &S, const KvCache &C, const NewRows &R, uint32_t *flags,
                          cudaStream_t stream);
cudaError_t launch_compact(const KvSeqs &S, const KvCache &C, const int32_t *path, int width,
                           const int32_t *accepted, int32_t *out_len, uint32_t *flags,
                           cudaStream_t stream);
cudaError_t launch_resize(const Pool &P, const int32_t *length, uint32_t *flags,
                          cudaStream_t stream);
size_t fork_workspace_bytes(int F);
cudaError_t launch_fork(const Pool &P, const KvCache &C, int32_t *ctx, const int32_t *src,
                        const int32_t *dst, int F, void *workspace, uint32_t *flags,
                        cudaStream_t stream);
}  // namespace sv

namespace {

using sv::kMaxNew;
using sv::kMaxSeqs;
constexpr int kMaxHeadDim = 256;
constexpr int kMaxPageSize = 65536;
constexpr int kMaxRowsY = 65535;  // blockIdx.y
constexpr int64_t kMaxPagePieces = 1 << 30;  // of 16 bytes: a page's copy counts them in 32 bits

spec_status map_cuda(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }

int kv_esize(spec_dtype d) {
  return d == SPEC_BF16 || d == SPEC_F16 ? 2 : (d == SPEC_F32 ? 4 : 0);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A stride of a dimension of n rows: rows apart, 16-byte aligned, and small
// enough that the byte offset of the last row stays in 64 bits.
bool stride_ok(int64_t stride, int64_t n, int head_dim, int esize) {
  if (n <= 1) return true;
  return stride >= head_dim && stride * esize % 16 == 0 && stride < (INT64_MAX >> 4) / n;
}

spec_status check_cache(const spec_kv_cache &c) {
  const int esize = kv_esize(c.dtype);
  if (esize == 0 || !c.k || !c.v || c.num_layers < 1 || c.num_pages < 1 || c.page_size < 1 ||
      c.page_size > kMaxPageSize || c.num_heads < 1 || c.head_dim < 1)
    return SPEC_ERR_INVALID_ARG;
  if (c.head_dim > kMaxHeadDim || c.head_dim * esize % 16 != 0 || !aligned16(c.k) ||
      !aligned16(c.v) || c.num_layers > kMaxRowsY / 2 || c.num_heads > 4096 ||
      static_cast<int64_t>(c.page_size) * c.num_heads * (c.head_dim * esize / 16) > kMaxPagePieces)
    return SPEC_ERR_UNSUPPORTED;
  const int64_t strides[8] = {c.k_layer_stride, c.k_page_stride, c.k_token_stride, c.k_head_stride,
                              c.v_layer_stride, c.v_page_stride, c.v_token_stride, c.v_head_stride};
  const int64_t sizes[4] = {c.num_layers, c.num_pages, c.page_size, c.num_heads};
  for (int i = 0; i < 8; ++i)
    if (!stride_ok(strides[i], sizes[i & 3], c.head_dim, esize)) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

bool table_ok(const spec_page_table &t, int page_size) {
  return t.table && t.max_pages >= 1 && t.ld >= t.max_pages &&
         static_cast<int64_t>(t.max_pages) * page_size < INT_MAX - 2 * kMaxNew;
}

sv::KvCache view(const spec_kv_cache &c) {
  const int e = kv_esize(c.dtype);
  sv::KvCache v;
  v.k = static_cast<char *>(c.k);
  v.v = static_cast<char *>(c.v);
  v.k_layer = c.k_layer_stride * e;
  v.k_page = c.k_page_stride * e;
  v.k_token = c.k_token_stride * e;
  v.k_head = c.k_head_stride * e;
  v.v_layer = c.v_layer_stride * e;
  v.v_page = c.v_page_stride * e;
  v.v_token = c.v_token_stride * e;
  v.v_head = c.v_head_stride * e;
  v.layers = c.num_layers;
  v.pages = c.num_pages;
  v.page_size = c.page_size;
  v.heads = c.num_heads;
  v.row_bytes = c.head_dim * e;
  return v;
}

sv::KvSeqs view(const spec_page_table &t, const int32_t *ctx, const int32_t *num_new, int B, int N) {
  sv::KvSeqs s;
  s.table = t.table;
  s.ld_table = t.ld;
  s.max_pages = t.max_pages;
  s.ctx = ctx;
  s.num_new = num_new;
  s.B = B;
  s.N = N;
  return s;
}

bool pool_ok(const spec_page_pool &p) {
  return p.page_table && p.page_count && p.ref_count && p.free_list && p.free_count &&
         p.max_pages >= 1 && p.ld_table >= p.max_pages && p.num_pages >= 1 && p.page_size >= 1 &&
         p.page_size <= kMaxPageSize && p.num_seqs <= kMaxSeqs &&
         static_cast<int64_t>(p.max_pages) * p.page_size < INT_MAX - 2 * kMaxNew &&
         static_cast<int64_t>(p.num_seqs) * p.max_pages < (1 << 30);
}

sv::Pool view(const spec_page_pool &p) {
  sv::Pool v;
  v.table = p.page_table;
  v.ld_table = p.ld_table;
  v.max_pages = p.max_pages;
  v.count = p.page_count;
  v.refs = p.ref_count;
  v.free_list = p.free_list;
  v.free_count = p.free_count;
  v.B = p.num_seqs;
  v.pages = p.num_pages;
  v.page_size = p.page_size;
  return v;
}

bool attention_sizes_ok(int B, int N, int Hq, int Hkv, int D, spec_dtype dtype) {
  const int e = kv_esize(dtype);
  return e != 0 && B >= 0 && N >= 1 && N <= kMaxNew && Hkv >= 1 && Hkv <= 4096 && Hq >= Hkv &&
         Hq <= 65536 && Hq % Hkv == 0 && D >= 1 && D <= kMaxHeadDim && D * e % 16 == 0 &&
         static_cast<int64_t>(B) * N < (1 << 28);
}

}  // namespace

extern "C" {

size_t spec_paged_attention_workspace_size(int B, int N, int num_q_heads, int num_kv_heads,
                                           int head_dim, spec_dtype dtype) {
  if (!attention_sizes_ok(B, N, num_q_heads, num_kv_heads, head_dim, dtype)) return 0;
  return sv::attention_workspace_bytes(N, num_q_heads / num_kv_heads, head_dim, dtype);
}

spec_status spec_paged_attention(
    const void *q, int64_t q_seq_stride, int64_t q_token_stride, int64_t q_head_stride,
    int num_q_heads, spec_kv_cache cache, spec_page_table pages, const int32_t *context_len,
    const int32_t *num_new, int B, int N, const uint64_t *tree_mask, int64_t mask_seq_stride,
    const int32_t *position, int64_t position_seq_stride, float scale, int window, int sinks,
    void *out, float *out_lse, uint32_t *out_flags, void *workspace, size_t workspace_bytes,
    spec_stream_t stream) {
  const int esize = kv_esize(cache.dtype);
  if (esize == 0 || B < 0 || N < 1 || N > kMaxNew || num_q_heads < 1 || !(scale > 0.f) ||
      !(scale * sv::kLog2e < INFINITY) || sinks < 0)
    return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (const spec_status s = check_cache(cache); s != SPEC_OK) return s;
  if (cache.num_layers != 1 || num_q_heads % cache.num_heads != 0 || !q || !out || !context_len ||
      !table_ok(pages, cache.page_size) || (window > 0 && tree_mask && !position) ||
      mask_seq_stride < 0 || position_seq_stride < 0)
    return SPEC_ERR_INVALID_ARG;
  if (!attention_sizes_ok(B, N, num_q_heads, cache.num_heads, cache.head_dim, cache.dtype))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !stride_ok(q_seq_stride, B, cache.head_dim, esize) ||
      !stride_ok(q_token_stride, N, cache.head_dim, esize) ||
      !stride_ok(q_head_stride, num_q_heads, cache.head_dim, esize))
    return SPEC_ERR_UNSUPPORTED;
  // pieces of a unit read its queries while others write its outputs
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(out);
  const uintptr_t q1 = q0 + (static_cast<uintptr_t>(B - 1) * (B > 1 ? q_seq_stride : 0) +
                             static_cast<uintptr_t>(N - 1) * (N > 1 ? q_token_stride : 0) +
                             static_cast<uintptr_t>(num_q_heads - 1) *
                                 (num_q_heads > 1 ? q_head_stride : 0) +
                             cache.head_dim) * esize;
  const uintptr_t o1 =
      o0 + static_cast<uintptr_t>(B) * N * num_q_heads * cache.head_dim * esize;
  if (q0 < o1 && o0 < q1) return SPEC_ERR_INVALID_ARG;
  const int group = num_q_heads / cache.num_heads;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 31u) != 0 ||
      workspace_bytes < sv::attention_workspace_bytes(N, group, cache.head_dim, cache.dtype))
    return SPEC_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  sv::AttnParams p = {};
  p.q = static_cast<const char *>(q);
  p.q_seq = q_seq_stride * esize;
  p.q_token = q_token_stride * esize;
  p.q_head = q_head_stride * esize;
  p.C = view(cache);
  p.S = view(pages, context_len, num_new, B, N);
  p.mask = tree_mask;
  p.mask_seq = mask_seq_stride;
  p.words = (N + 63) / 64;
  p.position = position;
  p.position_seq = position_seq_stride;
  p.G = group;
  p.D = cache.head_dim;
  p.scale = scale;
  p.scale_log2 = scale * sv::kLog2e;
  // a window that holds every place of a sequence is none
  const int places = pages.max_pages * cache.page_size + N;
  p.window = window > 0 && window < places ? window : 0;
  p.sinks = sinks;
  p.out = out;
  p.lse = out_lse;
  p.flags = out_flags;
  p.first_wait = sv::first_wait_cycles();
  if (out_flags) {
    const cudaError_t e = sv::launch_kv_flags(p.S, p.C, false, p.window, p.sinks, out_flags, st);
    if (e != cudaSuccess) return map_cuda(e);
  }
  return map_cuda(sv::launch_attention(p, cache.dtype, workspace, st));
}

spec_status spec_cache_append(
    const void *k_new, int64_t k_layer_stride, int64_t k_seq_stride, int64_t k_token_stride,
    int64_t k_head_stride, const void *v_new, int64_t v_layer_stride, int64_t v_seq_stride,
    int64_t v_token_stride, int64_t v_head_stride, spec_kv_cache cache, spec_page_table pages,
    const int32_t *context_len, const int32_t *num_new, int B, int N, uint32_t *out_flags,
    spec_stream_t stream) {
  if (B < 0 || N < 0 || N > kMaxNew || static_cast<int64_t>(B) * N >= (1 << 28))
    return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (const spec_status s = check_cache(cache); s != SPEC_OK) return s;
  if (!context_len || !table_ok(pages, cache.page_size) || (N > 0 && (!k_new || !v_new)))
    return SPEC_ERR_INVALID_ARG;
  const int e = kv_esize(cache.dtype), D = cache.head_dim;
  if (!aligned16(k_new) || !aligned16(v_new) || !stride_ok(k_layer_stride, cache.num_layers, D, e) ||
      !stride_ok(k_seq_stride, B, D, e) || !stride_ok(k_token_stride, N, D, e) ||
      !stride_ok(k_head_stride, cache.num_heads, D, e) ||
      !stride_ok(v_layer_stride, cache.num_layers, D, e) || !stride_ok(v_seq_stride, B, D, e) ||
      !stride_ok(v_token_stride, N, D, e) || !stride_ok(v_head_stride, cache.num_heads, D, e))
    return SPEC_ERR_UNSUPPORTED;
  sv::NewRows r;
  r.k = static_cast<const char *>(k_new);
  r.v = static_cast<const char *>(v_new);
  r.k_layer = k_layer_stride * e;
  r.k_seq = k_seq_stride * e;
  r.k_token = k_token_stride * e;
  r.k_head = k_head_stride * e;
  r.v_layer = v_layer_stride * e;
  r.v_seq = v_seq_stride * e;
  r.v_token = v_token_stride * e;
  r.v_head = v_head_stride * e;
  return map_cuda(sv::launch_append(view(pages, context_len, num_new, B, N), view(cache), r,
                                    out_flags, reinterpret_cast<cudaStream_t>(stream)));
}

spec_status spec_cache_compact(spec_kv_cache cache, spec_page_table pages,
                               const int32_t *context_len, const int32_t *path, int width,
                               const int32_t *num_accepted, int B, int32_t *out_context_len,
                               uint32_t *out_flags, spec_stream_t stream) {
  if (B < 0 || width < 1 || width > sv::kMaxPath) return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (const spec_status s = check_cache(cache); s != SPEC_OK) return s;
  if (!context_len || !path || !num_accepted || !out_context_len ||
      out_context_len == context_len || !table_ok(pages, cache.page_size))
    return SPEC_ERR_INVALID_ARG;
  return map_cuda(sv::launch_compact(view(pages, context_len, nullptr, B, 0), view(cache), path,
                                     width, num_accepted, out_context_len, out_flags,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

spec_status spec_cache_resize(spec_page_pool pool, const int32_t *length, uint32_t *out_flags,
                              spec_stream_t stream) {
  if (pool.num_seqs < 0) return SPEC_ERR_INVALID_ARG;
  if (pool.num_seqs == 0) return SPEC_OK;
  if (!pool_ok(pool) || !length) return SPEC_ERR_INVALID_ARG;
  return map_cuda(
      sv::launch_resize(view(pool), length, out_flags, reinterpret_cast<cudaStream_t>(stream)));
}

size_t spec_cache_fork_workspace_size(int F) {
  return F < 0 || F > kMaxSeqs ? 0 : sv::fork_workspace_bytes(F);
}

spec_status spec_cache_fork(spec_page_pool pool, spec_kv_cache cache, int32_t *context_len,
                            const int32_t *src, const int32_t *dst, int F, uint32_t *out_flags,
                            void *workspace, size_t workspace_bytes, spec_stream_t stream) {
  if (F < 0 || F > kMaxSeqs || pool.num_seqs < 0) return SPEC_ERR_INVALID_ARG;
  if (F == 0) return SPEC_OK;
  if (!pool_ok(pool) || !context_len || !src || !dst || !workspace ||
      (reinterpret_cast<uintptr_t>(workspace) & 3u) != 0 ||
      workspace_bytes < sv::fork_workspace_bytes(F))
    return SPEC_ERR_INVALID_ARG;
  if (const spec_status s = check_cache(cache); s != SPEC_OK) return s;
  if (cache.num_pages != pool.num_pages || cache.page_size != pool.page_size)
    return SPEC_ERR_INVALID_ARG;
  return map_cuda(sv::launch_fork(view(pool), view(cache), context_len, src, dst, F, workspace,
                                  out_flags, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
