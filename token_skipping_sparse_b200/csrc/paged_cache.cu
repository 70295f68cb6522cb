// paged_cache.cu -- filling the paged key/value cache and evicting from it.
#include "host.hpp"
#include "paged.cuh"
#include "rowops.cuh"

namespace spts {
namespace {

// Last b with cu[b] <= t: the sequence of packed row t.
__device__ __forceinline__ int owner_of(const int32_t *cu, int B, int t) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------ append
// One CTA per new token: K and V rows in 16-byte pieces, K turned by RoPE in
// fp32 (pair (i, i + d/2), so a thread takes the two pieces that pair up).
__global__ void __launch_bounds__(128)
    cache_append_kernel(PagedView c, const __nv_bfloat16 *__restrict__ k_new, int64_t k_stride,
                        const __nv_bfloat16 *__restrict__ v_new, int64_t v_stride, const int32_t *__restrict__ cu,
                        int T, const int32_t *__restrict__ pos, const __grid_constant__ RopeFreqs f,
                        uint32_t *status) {
  const int row = blockIdx.x;
  if (row == 0) check_sequences(c, cu, T, status);
  if (row >= __ldg(cu + c.B)) return;
  const int b = owner_of(cu, c.B, row);
  int first, n;
  packed_span(cu, T, b, nullptr, first, n);
  const int t = paged_len(c, b, nullptr) - n + (row - first);
  if (t < 0 || row < first || row >= first + n) {
    if (threadIdx.x == 0 && t < 0) raise_status(status, SPTS_DEV_BADINDEX, kSiteSlot, static_cast<uint32_t>(row));
    return;
  }
  const int page = paged_page(c.table, c.table_stride, c.num_pages, b, t >> c.page_shift,
                              threadIdx.x == 0 ? status : nullptr);
  if (page < 0) return;
  const int64_t at = paged_offset(c, page, t, 0);
  const uint4 *ks = reinterpret_cast<const uint4 *>(k_new + row * k_stride);
  const uint4 *vs = reinterpret_cast<const uint4 *>(v_new + row * v_stride);
  uint4 *kd = reinterpret_cast<uint4 *>(c.k + at), *vd = reinterpret_cast<uint4 *>(c.v + at);
  const int vecs = c.Hkv * c.d / 8;
  for (int i = threadIdx.x; i < vecs; i += blockDim.x) vd[i] = vs[i];
  if (pos == nullptr) {
    for (int i = threadIdx.x; i < vecs; i += blockDim.x) kd[i] = ks[i];
    return;
  }
  const int32_t p = __ldg(pos + row);
  const int half = c.d / 16;  // pieces of half a head
  for (int i = threadIdx.x; i < vecs / 2; i += blockDim.x) {
    const int h = i / half, j = i % half, lo = h * 2 * half + j;
    uint4 a = ks[lo], e = ks[lo + half];
    __nv_bfloat16 *pa = reinterpret_cast<__nv_bfloat16 *>(&a), *pe = reinterpret_cast<__nv_bfloat16 *>(&e);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      float cs, sn;
      rope_cos_sin(p, f, j * 8 + u, &cs, &sn);
      const float x = __bfloat162float(pa[u]), y = __bfloat162float(pe[u]);
      pa[u] = __float2bfloat16(x * cs - y * sn);
      pe[u] = __float2bfloat16(y * cs + x * sn);
    }
    kd[lo] = a;
    kd[lo + half] = e;
  }
}

// ------------------------------------------------------------------ evict: selection
constexpr int SEL_THREADS = 1024;

__device__ __forceinline__ uint32_t weight_key(float f) {
  uint32_t b = __float_as_uint(f);
  if (b == 0x80000000u) b = 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Exclusive scan of one value per thread of the CTA; *total = the sum.
__device__ __forceinline__ uint32_t scan_excl(uint32_t v, uint32_t *warp_tot, uint32_t *total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_tot[w] = x;
  __syncthreads();
  if (w == 0) {
    const uint32_t t = warp_tot[lane];
    uint32_t u = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, u, o);
      if (lane >= o) u += y;
    }
    warp_tot[lane] = u - t;
    if (lane == 31) *total = u;
  }
  __syncthreads();
  const uint32_t r = warp_tot[w] + x - v;
  __syncthreads();
  return r;
}

// One CTA per weight row (sequence, KV head or all heads): radix select of
// the kept tokens among the free slots [sink, L - recent) by 8-bit digits,
// compaction in slot order, then the weights of the kept tokens in tiles
// (each tile read before it is written, and never over a later tile's
// source, so weights_out may be weights).
__global__ void __launch_bounds__(SEL_THREADS) evict_select_kernel(PagedView c, EvictArgs e) {
  __shared__ uint32_t hist[256], warp_tot[32], s_total, s_digit, s_rem;
  const int row = blockIdx.x, b = row / e.Hs, tid = threadIdx.x;
  const int L = paged_len(c, b, tid == 0 ? e.status : nullptr);
  const float *w = e.weights + row * e.w_stride;
  int32_t *kept = e.kept + row * e.kept_stride;
  const int new_len = min(L, e.keep);
  if (L <= e.keep) {
    for (int t = tid; t < L; t += SEL_THREADS) kept[t] = t;
  } else {
    const int lo = e.sink, hi = L - e.recent, k_free = e.keep - e.sink - e.recent;
    uint32_t T = 0xffffffffu, rem = 0;
    if (k_free > 0) {
      uint32_t prefix = 0, mask = 0;
      rem = k_free;
      for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int i = lo + tid; i < hi; i += SEL_THREADS) {
          const uint32_t key = weight_key(w[i]);
          if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (tid == 0) {
          uint32_t above = 0;
          int d = 255;
          for (; d > 0 && above + hist[d] < rem; --d) above += hist[d];
          s_digit = d;
          s_rem = rem - above;
        }
        __syncthreads();
        prefix |= s_digit << shift;
        mask |= 255u << shift;
        rem = s_rem;
        __syncthreads();
      }
      T = prefix;
    }
    for (int t = tid; t < e.sink; t += SEL_THREADS) kept[t] = t;
    for (int t = tid; t < e.recent; t += SEL_THREADS) kept[e.keep - e.recent + t] = hi + t;
    if (k_free > 0) {
      uint32_t done_gt = 0, done_eq = 0;
      for (int base = lo; base < hi; base += SEL_THREADS) {
        const int i = base + tid;
        const float f = i < hi ? w[i] : 0.f;
        if (!isfinite(f)) raise_status(e.status, SPTS_DEV_BADINDEX, 0xA5u, static_cast<uint32_t>(i));
        const uint32_t key = weight_key(f);
        const uint32_t gt = i < hi && key > T, eq = i < hi && key == T;
        const uint32_t x = scan_excl(gt | (eq << 16), warp_tot, &s_total);
        const uint32_t before_eq = done_eq + (x >> 16), before = done_gt + (x & 0xffffu) + min(before_eq, rem);
        if (gt || (eq && before_eq < rem)) kept[e.sink + before] = i;
        done_gt += s_total & 0xffffu;
        done_eq += s_total >> 16;
        __syncthreads();
      }
    }
  }
  for (int64_t t = new_len + tid; t < e.kept_stride; t += SEL_THREADS) kept[t] = -1;
  __syncthreads();
  float *out = e.weights_out + row * e.w_out_stride;
  for (int base = 0; base < new_len; base += SEL_THREADS) {
    const int t = base + tid;
    const float f = t < new_len ? w[kept[t]] : 0.f;
    __syncthreads();
    if (t < new_len) out[t] = f;
  }
  __syncthreads();
  for (int64_t t = new_len + tid; t < e.w_out_stride; t += SEL_THREADS) out[t] = 0.f;
}

// ------------------------------------------------------------------ evict: moving the rows
// One CTA per (sequence, KV head) of K or of V walks the kept slots in order,
// a tile at a time: it reads the tile's rows, waits for all its threads, and
// writes them.  kept[t] >= t and ascending, so in place a tile's writes never
// reach the source of a later tile.
constexpr int MOVE_THREADS = 256;

__global__ void __launch_bounds__(MOVE_THREADS) evict_move_kernel(PagedView c, EvictArgs e) {
  const int b = blockIdx.x / c.Hkv, g = blockIdx.x % c.Hkv, tid = threadIdx.x;
  uint32_t *status = tid == 0 ? e.status : nullptr;
  __nv_bfloat16 *pages = blockIdx.y ? c.v : c.k;
  const int n = min(paged_len(c, b, status), e.keep);
  if (g == 0 && blockIdx.y == 0 && tid == 0) e.new_lens[b] = n;
  const int32_t *kept = e.kept + (static_cast<int64_t>(b) * e.Hs + (e.Hs == 1 ? 0 : g)) * e.kept_stride;
  const int vecs = c.d / 8, per = MOVE_THREADS / vecs, r = tid / vecs, x = tid % vecs;
  for (int base = 0; base < n; base += per) {
    const int t = base + r;
    uint4 val;
    bool ok = false;
    if (t < n) {
      const int from = kept[t];
      const int page = paged_page(c.table, c.table_stride, c.num_pages, b, from >> c.page_shift, e.status);
      if (page >= 0) {
        val = reinterpret_cast<const uint4 *>(pages + paged_offset(c, page, from, g))[x];
        ok = true;
      }
    }
    __syncthreads();
    if (ok) {
      const int entry = t >> c.page_shift;
      const int page = entry < e.dst_max_pages
                           ? paged_page(e.dst_table, e.dst_stride, c.num_pages, b, entry, e.status)
                           : -1;
      if (page >= 0) reinterpret_cast<uint4 *>(pages + paged_offset(c, page, t, g))[x] = val;
      else if (entry >= e.dst_max_pages) raise_status(e.status, SPTS_DEV_BADINDEX, kSiteSlot, t);
    }
  }
}

}  // namespace

spts_status launch_cache_append(const PagedView &c, const void *k_new, int64_t k_stride, const void *v_new,
                                int64_t v_stride, const int32_t *cu, int64_t T, const int32_t *pos, double theta,
                                uint32_t *status, cudaStream_t s) {
  if (T == 0) return SPTS_OK;
  RopeFreqs f;
  if (pos) fill_rope_freqs(&f, c.d, theta);
  cache_append_kernel<<<static_cast<unsigned>(T), 128, 0, s>>>(
      c, static_cast<const __nv_bfloat16 *>(k_new), k_stride, static_cast<const __nv_bfloat16 *>(v_new), v_stride, cu,
      static_cast<int>(T), pos, f, status);
  note_launch();
  SPTS_CUDA_TRY(cudaGetLastError());
  return SPTS_OK;
}

spts_status launch_cache_evict(const PagedView &c, const EvictArgs &e, cudaStream_t s) {
  evict_select_kernel<<<static_cast<unsigned>(c.B) * e.Hs, SEL_THREADS, 0, s>>>(c, e);
  note_launch();
  SPTS_CUDA_TRY(cudaGetLastError());
  evict_move_kernel<<<dim3(static_cast<unsigned>(c.B) * c.Hkv, 2), MOVE_THREADS, 0, s>>>(c, e);
  note_launch();
  SPTS_CUDA_TRY(cudaGetLastError());
  return SPTS_OK;
}

}  // namespace spts
