// The paged key-value cache as the kernels see it, and the flag rules shared
// by the operators on it.
#pragma once

#include <atomic>

#include "common.cuh"

namespace sv {

constexpr int kMaxNew = 4096;          // new tokens of a sequence in a call
constexpr int kMaxPath = kMaxNew + 1;  // entries of an accepted path
constexpr int kMaxSeqs = 4096;         // of a pool, and of the forks of a call

// One layer's keys and values start at k and v; strides are in bytes.
struct KvCache {
  char *k, *v;
  long long k_layer, k_page, k_token, k_head;
  long long v_layer, v_page, v_token, v_head;
  int layers, pages, page_size, heads, row_bytes;
};

// Page tables and lengths of the sequences of a call.
struct KvSeqs {
  const int32_t *table;
  long long ld_table;
  int max_pages;
  const int32_t *ctx;      // tokens of each sequence before the new ones
  const int32_t *num_new;  // may be NULL: N new tokens each
  int B, N;
};

// New keys and values of an append; strides in bytes.
struct NewRows {
  const char *k, *v;
  long long k_layer, k_seq, k_token, k_head;
  long long v_layer, v_seq, v_token, v_head;
};

// The page tables and the free list of a page pool.
struct Pool {
  int32_t *table;
  long long ld_table;
  int max_pages;
  int32_t *count, *refs, *free_list, *free_count;
  int B, pages, page_size;
};

// New tokens of sequence b, clamped into [0, N].
__device__ __forceinline__ int seq_new(const KvSeqs &S, int b) {
  return S.num_new ? min(max(__ldg(S.num_new + b), 0), S.N) : S.N;
}

// Whether ctx tokens and n new ones fit the sequence's row of the page table.
// The host keeps max_pages * page_size + N below 2^31.
__device__ __forceinline__ bool seq_fits(const KvSeqs &S, const KvCache &C, int ctx, int n) {
  return ctx >= 0 && ctx <= S.max_pages * C.page_size - n;
}

__device__ __forceinline__ int page_at(const KvSeqs &S, int b, int index) {
  return __ldg(S.table + static_cast<long long>(b) * S.ld_table + index);
}
__device__ __forceinline__ bool page_ok(const KvCache &C, int page) {
  return static_cast<unsigned>(page) < static_cast<unsigned>(C.pages);
}

// Flags of each sequence: SPEC_FLAG_BAD_LENGTH (num_new outside [0, N], or
// tokens that do not fit the table row) and SPEC_FLAG_BAD_PAGE (a page id
// outside the cache among the pages that are looked at: those of the new tokens
// alone, or all but those behind the sinks that a window (0: none) hides from every
// new token).  One launch.
cudaError_t launch_kv_flags(const KvSeqs &S, const KvCache &C, bool new_only, int window, int sinks,
                            uint32_t *flags, cudaStream_t stream);

// Launch of a kernel with much dynamic shared memory.  It is allowed the `most`
// that any call of it uses once per device (done: a bit each): the call for it costs
// a good part of a launch's host time, and a thread that allowed less for its own
// call would have another's launch refused.  A context that has forgotten it is told
// again.
template <typename... KP, typename... A>
cudaError_t launch_large(void (*kernel)(KP...), std::atomic<uint64_t> &done, int most, dim3 grid,
                         int threads, int smem, cudaStream_t stream, const A &...args) {
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  for (;;) {
    const bool told = (done.load(std::memory_order_relaxed) & bit) != 0;
    if (!told) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (e != cudaSuccess) return e;
      done.fetch_or(bit, std::memory_order_relaxed);
    }
    kernel<<<grid, threads, smem, stream>>>(args...);
    e = cudaGetLastError();
    if (e != cudaErrorInvalidValue || !told) return e;
    done.fetch_and(~bit, std::memory_order_relaxed);
  }
}

// Launch with programmatic stream serialisation: the kernel may start while
// the previous one on the stream drains, and waits for it at its own
// griddepcontrol.wait.
template <typename... KP, typename... A>
cudaError_t launch_behind(void (*kernel)(KP...), dim3 grid, int threads, size_t smem,
                          cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace sv
