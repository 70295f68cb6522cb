// paged.cuh -- the paged key/value cache as the kernels see it (page
// addressing, the lengths and offsets that live on the device) and the
// launchers of the kernels that fill it, attend over it and evict from it.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <utility>

#include "host.hpp"
#include "status.cuh"

namespace spts {

struct PagedView {
  __nv_bfloat16 *k, *v;
  const int32_t *table;
  const int32_t *lens;
  int64_t page_stride;   // elements between pages
  int64_t table_stride;  // entries between rows of the table
  int num_pages;
  int page_shift;        // page_size = 1 << page_shift
  int B, max_pages;
  int Hkv, d;
};

// Kernel-specific sites of the flags raised here.
constexpr uint32_t kSitePage = 0xA1u;    // page number out of range
constexpr uint32_t kSiteLen = 0xA2u;     // sequence length out of range
constexpr uint32_t kSiteOffset = 0xA3u;  // packed offsets out of range or descending
constexpr uint32_t kSiteSlot = 0xA4u;    // a token without a slot
constexpr uint32_t kSiteWeight = 0xA5u;  // a weight that is not finite

// Cached tokens of sequence b, clamped to what its table row can hold.
__device__ __forceinline__ int paged_len(const PagedView &c, int b, uint32_t *status) {
  const int len = __ldg(c.lens + b), cap = c.max_pages << c.page_shift;
  const int ok = min(max(len, 0), cap);
  if (ok != len) raise_status(status, SPTS_DEV_BADINDEX, kSiteLen, static_cast<uint32_t>(b));
  return ok;
}

// First packed row and number of rows of sequence b, clamped to [0, T].
__device__ __forceinline__ void packed_span(const int32_t *cu, int T, int b, uint32_t *status, int &first, int &n) {
  const int lo = __ldg(cu + b), hi = __ldg(cu + b + 1);
  first = min(max(lo, 0), T);
  n = max(min(max(hi, 0), T) - first, 0);
  if (lo < 0 || hi > T || hi < lo || (b == 0 && lo != 0))
    raise_status(status, SPTS_DEV_BADINDEX, kSiteOffset, static_cast<uint32_t>(b));
}

// Flags what is wrong with the lengths and offsets; by one CTA of a launch.
__device__ __forceinline__ void check_sequences(const PagedView &c, const int32_t *cu, int T, uint32_t *status) {
  for (int b = threadIdx.x; b < c.B; b += blockDim.x) {
    int first, n;
    packed_span(cu, T, b, status, first, n);
    paged_len(c, b, status);
  }
}

// Page number of entry `e` of row b of a page table, or -1 (flag raised) when
// it names no page.
__device__ __forceinline__ int paged_page(const int32_t *table, int64_t stride, int num_pages, int b, int e,
                                          uint32_t *status) {
  const int page = __ldg(table + b * stride + e);
  if (static_cast<uint32_t>(page) < static_cast<uint32_t>(num_pages)) return page;
  raise_status(status, SPTS_DEV_BADINDEX, kSitePage, static_cast<uint32_t>(page));
  return -1;
}

// Element offset of slot t's row of KV head g inside page `page`.
__device__ __forceinline__ int64_t paged_offset(const PagedView &c, int page, int t, int g) {
  return page * c.page_stride + (static_cast<int64_t>(t & ((1 << c.page_shift) - 1)) * c.Hkv + g) * c.d;
}

// Allows a kernel `bytes` of dynamic shared memory, once per device.
template <auto Kernel>
spts_status allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done[4];
  int dev = 0;
  SPTS_CUDA_TRY(cudaGetDevice(&dev));
  const uint64_t bit = uint64_t(1) << (dev & 63);
  std::atomic<uint64_t> &word = done[(dev >> 6) & 3];
  if (dev < 256 && (word.load(std::memory_order_acquire) & bit)) return SPTS_OK;
  SPTS_CUDA_TRY(cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)));
  word.fetch_or(bit, std::memory_order_release);
  return SPTS_OK;
}

// Launches a kernel that may start while the one before it on the stream still
// runs, and waits for it itself (griddepcontrol.wait).
template <typename... Want, typename... Args>
spts_status launch_behind(void (*kernel)(Want...), dim3 grid, int threads, cudaStream_t s, size_t smem,
                          Args &&...args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  SPTS_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...));
  note_launch();
  return SPTS_OK;
}

spts_status launch_cache_append(const PagedView &c, const void *k_new, int64_t k_stride, const void *v_new,
                                int64_t v_stride, const int32_t *cu, int64_t T, const int32_t *pos, double theta,
                                uint32_t *status, cudaStream_t s);

struct PagedAttnArgs {
  const void *q;
  int64_t q_stride;
  const int32_t *cu;
  int64_t T;
  int Hq;
  float scale;
  void *o;
  int64_t o_stride;
  float *lse;      // [T, Hq]; needed with weights
  float *weights;  // [B, Hs, w_stride] or NULL
  int Hs;
  int64_t w_stride;
  uint32_t *status;
  void *scratch;     // paged_attn_scratch_bytes(...)
  float *w_scratch;  // paged_weights_scratch(...) floats, or NULL
  float *scores;     // paged_scores_bytes(...), or NULL
};
// TMA maps of q (box: 64 columns x G heads x `tokens`) and of K or V pages (64
// columns x one head x the rows of a page, at most 128).
spts_status paged_q_map(const PagedView &c, const PagedAttnArgs &a, int tokens, CUtensorMap *q);
spts_status paged_kv_map(const PagedView &c, const void *pages, CUtensorMap *map);
size_t paged_attn_scratch_bytes(int B, int64_t T, int64_t slots, int Hq, int Hkv, int d);
spts_status launch_paged_attention(const PagedView &c, const PagedAttnArgs &a, cudaStream_t s);
size_t paged_scores_bytes(int B, int64_t T, int64_t slots, int Hq, int Hkv);
// Adds to a.weights what the attention that left a.lse gave each slot: from
// the scores that it left too, or from a second product.
spts_status launch_stored_weights(const PagedView &c, const PagedAttnArgs &a, int64_t score_stride, cudaStream_t s);
size_t paged_weights_scratch(int B, int64_t slots, int Hkv, int Hs);
spts_status launch_paged_weights(const PagedView &c, const PagedAttnArgs &a, const CUtensorMap &tmK, cudaStream_t s);

struct EvictArgs {
  const float *weights;
  int Hs;
  int64_t w_stride;
  int keep, sink, recent;
  const int32_t *dst_table;
  int dst_max_pages;
  int64_t dst_stride;
  float *weights_out;
  int64_t w_out_stride;
  int32_t *new_lens;
  int32_t *kept;        // [B, Hs, kept_stride], kept_stride >= min(keep, slots of a table row)
  int64_t kept_stride;
  uint32_t *status;
};
spts_status launch_cache_evict(const PagedView &c, const EvictArgs &e, cudaStream_t s);

}  // namespace spts
