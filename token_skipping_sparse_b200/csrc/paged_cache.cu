// paged_cache.cu -- filling the paged key/value cache and evicting from it.
// Everything here is bound by the bytes it moves, or for small calls by the
// chain of dependent loads (offset, length, page, row); there is no arithmetic
// to speak of.
#include "host.hpp"
#include "paged.cuh"
#include "paged_plan.hpp"
#include "rowops.cuh"
#include "sm100.cuh"

namespace spts {
namespace {

constexpr int MAX_SEQ = 1024;

// ------------------------------------------------------------------ append
// A thread takes one 16-byte piece of the lower half of a token's heads and
// the piece d/2 further on that RoPE pairs it with, for K and V of `heads`
// heads: the angles are found once for all of them, and all loads of four
// heads are in flight together.  RoPE in fp32, rounded once.
constexpr int APPEND_THREADS = 256;

template <int D>
__global__ void __launch_bounds__(APPEND_THREADS)
    cache_append_kernel(PagedView c, const __nv_bfloat16 *__restrict__ k_new, int64_t k_stride,
                        const __nv_bfloat16 *__restrict__ v_new, int64_t v_stride, const int32_t *__restrict__ cu,
                        int T, const int32_t *__restrict__ pos, int heads, const __grid_constant__ RopeFreqs f,
                        uint32_t *status) {
  constexpr int HALF = D / 16, TOKENS = APPEND_THREADS / HALF;  // pieces of half a head; tokens of a CTA
  __shared__ int offsets[MAX_SEQ + 1];
  if (blockIdx.x == 0 && blockIdx.y == 0) check_sequences(c, cu, T, status);
  for (int i = threadIdx.x; i <= c.B; i += APPEND_THREADS) offsets[i] = __ldg(cu + i);
  __syncthreads();
  const int row = blockIdx.x * TOKENS + threadIdx.x / HALF, j = threadIdx.x % HALF;
  if (row >= min(T, offsets[c.B])) return;
  int b = 0, end = c.B;  // the last sequence that begins at or before the row
  while (end - b > 1) {
    const int mid = (b + end) >> 1;
    if (offsets[mid] <= row) b = mid;
    else end = mid;
  }
  int first, n;
  packed_span(cu, T, b, nullptr, first, n);
  if (row < first || row >= first + n) return;
  uint32_t *flag = j == 0 && blockIdx.y == 0 ? status : nullptr;
  const int t = paged_len(c, b, nullptr) - n + (row - first);
  if (t < 0) {
    raise_status(flag, SPTS_DEV_BADINDEX, kSiteSlot, static_cast<uint32_t>(row));
    return;
  }
  const int page = paged_page(c.table, c.table_stride, c.num_pages, b, t >> c.page_shift, flag);
  if (page < 0) return;
  float cs[8], sn[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    cs[u] = 1.f;
    sn[u] = 0.f;
  }
  if (pos != nullptr) {
    const int32_t p = __ldg(pos + row);
#pragma unroll
    for (int u = 0; u < 8; ++u) rope_cos_sin(p, f, j * 8 + u, &cs[u], &sn[u]);
  }
  const int h0 = blockIdx.y * heads, h1 = min(h0 + heads, c.Hkv);
  const int64_t at = paged_offset(c, page, t, 0);
  const uint4 *ks = reinterpret_cast<const uint4 *>(k_new + row * k_stride) + j;
  const uint4 *vs = reinterpret_cast<const uint4 *>(v_new + row * v_stride) + j;
  uint4 *kd = reinterpret_cast<uint4 *>(c.k + at) + j, *vd = reinterpret_cast<uint4 *>(c.v + at) + j;
  for (int h = h0; h < h1; h += 4) {
    uint4 kl[4], kh[4], vl[4], vh[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (h + u < h1) {
        const int o = (h + u) * 2 * HALF;
        kl[u] = __ldg(ks + o);
        kh[u] = __ldg(ks + o + HALF);
        vl[u] = __ldg(vs + o);
        vh[u] = __ldg(vs + o + HALF);
      }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (h + u < h1) {
        const int o = (h + u) * 2 * HALF;
        vd[o] = vl[u];
        vd[o + HALF] = vh[u];
        if (pos != nullptr) {
          uint32_t *lo = reinterpret_cast<uint32_t *>(&kl[u]), *hi = reinterpret_cast<uint32_t *>(&kh[u]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x0 = __uint_as_float(lo[e] << 16), x1 = __uint_as_float(lo[e] & 0xffff0000u);
            const float y0 = __uint_as_float(hi[e] << 16), y1 = __uint_as_float(hi[e] & 0xffff0000u);
            lo[e] = pack_bf16x2(x0 * cs[2 * e] - y0 * sn[2 * e], x1 * cs[2 * e + 1] - y1 * sn[2 * e + 1]);
            hi[e] = pack_bf16x2(y0 * cs[2 * e] + x0 * sn[2 * e], y1 * cs[2 * e + 1] + x1 * sn[2 * e + 1]);
          }
        }
        kd[o] = kl[u];
        kd[o + HALF] = kh[u];
      }
  }
}

// ------------------------------------------------------------------ evict: selection
// One cluster of up to 8 CTAs per weight row (sequence, KV head or all heads).
// The free slots [sink, L - recent) are shared out in contiguous slices, each
// kept in its CTA's shared memory as order-preserving keys, so the weights are
// read once.  Radix select with digits of 11, 11 and 10 bits: every CTA
// histograms its slice and adds the bins that are not empty to the totals of
// every CTA through distributed shared memory (reading all the others' 2048
// bins instead took 9000 cycles a digit, with the rest 24 us for a row of
// 32768); each finds the bin of the last kept key.  Then each warp counts
// the keys above and at the threshold in its part of the slice, and writes its
// kept slots behind those of the warps and CTAs before it: ascending, equal
// weights to the lower slot, no atomics whose order matters.
constexpr int SEL_THREADS = 1024;
constexpr int SEL_BINS = 2048;
constexpr int SEL_MAX_KEYS = 49152;  // keys a CTA can hold: 192 KB
constexpr int SEL_MAX_CLUSTER = 8;

__device__ __forceinline__ uint32_t weight_key(float f) {
  uint32_t b = __float_as_uint(f);
  if (b == 0x80000000u) b = 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Sum of v[0..w) (32 entries in shared memory), by a whole warp.
__device__ __forceinline__ uint32_t sum_below(const uint32_t *v, int w) {
  const int lane = threadIdx.x & 31;
  return __reduce_add_sync(0xffffffffu, lane < w ? v[lane] : 0u);
}

__device__ __forceinline__ void add_cluster(const uint32_t *p, uint32_t cta, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(cluster_addr(p, cta)), "r"(v) : "memory");
}

__device__ __forceinline__ uint32_t ld_cluster(const uint32_t *p, uint32_t cta) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(p, cta)) : "memory");
  return v;
}

__global__ void __launch_bounds__(SEL_THREADS) evict_select_kernel(PagedView c, EvictArgs e, int ctas, int max_keys) {
  extern __shared__ uint32_t keys[];  // [max_keys]
  __shared__ uint32_t hist[SEL_BINS], all[3][SEL_BINS];  // this CTA's digit; the cluster's, per digit
  __shared__ uint32_t warp_gt[32], warp_eq[32], totals[2], s_digit, s_rem;
  const int row = blockIdx.x / ctas, rank = blockIdx.x % ctas, b = row / e.Hs, tid = threadIdx.x;
  const int lane = tid & 31, w = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int L = paged_len(c, b, tid == 0 && rank == 0 ? e.status : nullptr);
  const float *wt = e.weights + row * e.w_stride;
  int32_t *kept = e.kept + row * e.kept_stride;
  for (int64_t t = min(L, e.keep) + rank * SEL_THREADS + tid; t < e.kept_stride; t += ctas * SEL_THREADS) kept[t] = -1;
  if (L <= e.keep) {
    for (int t = rank * SEL_THREADS + tid; t < L; t += ctas * SEL_THREADS) kept[t] = t;
    return;  // all CTAs of the cluster
  }
  const int lo = e.sink, hi = L - e.recent, k_free = e.keep - e.sink - e.recent;
  if (rank == 0)
    for (int t = tid; t < e.sink; t += SEL_THREADS) kept[t] = t;
  if (rank == ctas - 1)
    for (int t = tid; t < e.recent; t += SEL_THREADS) kept[e.keep - e.recent + t] = hi + t;
  if (k_free == 0) return;
  const int slice = (((hi - lo) + ctas - 1) / ctas + 31) & ~31;
  const int s0 = min(lo + rank * slice, hi), n = min(slice, hi - s0);  // this CTA's slots [s0, s0 + n)
  const bool cached = slice <= max_keys;
  auto key_at = [&](int i) -> uint32_t { return cached ? keys[i] : weight_key(__ldg(wt + s0 + i)); };

  for (int i = tid; i < SEL_BINS; i += SEL_THREADS) hist[i] = all[0][i] = all[1][i] = all[2][i] = 0;
  __syncthreads();
  cluster_arrive_all();  // the totals are ready to be added to
  for (int i = tid; i < n; i += SEL_THREADS) {
    const float f = __ldg(wt + s0 + i);
    if (!isfinite(f)) raise_status(e.status, SPTS_DEV_BADINDEX, kSiteWeight, static_cast<uint32_t>(s0 + i));
    const uint32_t key = weight_key(f);
    if (cached) keys[i] = key;
    atomicAdd(&hist[key >> 21], 1u);
  }
  cluster_wait_all();
  uint32_t prefix = 0, mask = 0, rem = k_free;
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10, shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    __syncthreads();
    for (int i = tid; i < SEL_BINS; i += SEL_THREADS) {
      const uint32_t count = hist[i];
      if (count == 0) continue;
      hist[i] = 0;
      for (int r = 0; r < ctas; ++r) add_cluster(&all[pass][i], r, count);
    }
    cluster_sync_all();
    // thread tid has the bins top and top - 1, counted from the highest
    const int top = (1 << bits) - 1 - 2 * tid;
    const uint32_t c0 = top >= 0 ? all[pass][top] : 0u, c1 = top >= 0 ? all[pass][top - 1] : 0u;
    uint32_t incl = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_gt[w] = incl;
    __syncthreads();
    const uint32_t above = sum_below(warp_gt, w) + incl - c0 - c1;  // keys in higher bins
    if (above < rem && rem <= above + c0) {
      s_digit = top;
      s_rem = rem - above;
    } else if (above + c0 < rem && rem <= above + c0 + c1) {
      s_digit = top - 1;
      s_rem = rem - above - c0;
    }
    __syncthreads();
    prefix |= s_digit << shift;
    mask |= ((1u << bits) - 1u) << shift;
    rem = s_rem;
    if (pass < 2) {
      const int next = pass == 0 ? 10 : 0;
      const uint32_t last = pass == 0 ? 2047u : 1023u;
      for (int i = tid; i < n; i += SEL_THREADS) {
        const uint32_t key = key_at(i);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> next) & last], 1u);
      }
    }
  }
  const uint32_t T = prefix;  // keep what is above, and the first `rem` equal ones
  const int part = ((n + 31) / 32 + 31) & ~31, w0 = min(w * part, n), w1 = min(w0 + part, n);
  uint32_t gt = 0, eq = 0;
  for (int i = w0; i < w1; i += 32) {
    const uint32_t key = i + lane < w1 ? key_at(i + lane) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && key > T));
    eq += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && key == T));
  }
  if (lane == 0) {
    warp_gt[w] = gt;
    warp_eq[w] = eq;
  }
  __syncthreads();
  uint32_t gt0 = sum_below(warp_gt, w), eq0 = sum_below(warp_eq, w);
  if (tid == SEL_THREADS - 1) {
    totals[0] = gt0 + gt;
    totals[1] = eq0 + eq;
  }
  cluster_sync_all();
  for (int r = 0; r < rank; ++r) {
    gt0 += ld_cluster(&totals[0], r);
    eq0 += ld_cluster(&totals[1], r);
  }
  for (int i = w0; i < w1; i += 32) {
    const uint32_t key = i + lane < w1 ? key_at(i + lane) : 0u;
    const bool is_gt = i + lane < w1 && key > T, is_eq = i + lane < w1 && key == T;
    const uint32_t bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t g = gt0 + __popc(bg & below), q = eq0 + __popc(be & below);
    if (is_gt || (is_eq && q < rem)) kept[e.sink + g + min(q, rem)] = s0 + i + lane;
    gt0 += __popc(bg);
    eq0 += __popc(be);
  }
  cluster_sync_all();  // no CTA leaves while another may read its shared memory
}

// ------------------------------------------------------------------ evict: moving the rows
__device__ __forceinline__ int64_t dst_offset(const PagedView &c, const EvictArgs &e, int b, int t, int g) {
  const int entry = t >> c.page_shift;
  if (entry >= e.dst_max_pages) {
    raise_status(e.status, SPTS_DEV_BADINDEX, kSiteSlot, static_cast<uint32_t>(t));
    return -1;
  }
  const int page = paged_page(e.dst_table, e.dst_stride, c.num_pages, b, entry, e.status);
  return page < 0 ? -1 : paged_offset(c, page, t, g);
}
// The kept slots come from the caller's workspace: one that is none (two calls
// at once with one workspace) is flagged, and nothing is read outside the rows.
__device__ __forceinline__ int64_t src_offset(const PagedView &c, const EvictArgs &e, int b, int from, int g) {
  if (!paged_has_slot(from, c.max_pages, c.page_shift)) {
    raise_status(e.status, SPTS_DEV_BADINDEX, kSiteSlot, static_cast<uint32_t>(from));
    return -1;
  }
  const int page = paged_page(c.table, c.table_stride, c.num_pages, b, from >> c.page_shift, e.status);
  return page < 0 ? -1 : paged_offset(c, page, from, g);
}

constexpr int MOVE_THREADS = 256;
constexpr int MOVE_ROWS = 4;    // rows of a thread that are in flight together
constexpr int COPY_ROWS = 128;  // rows of a CTA

// The weights of one row's kept tokens, then zeros; in place too: a tile of
// TILE entries is read before it is written, kept[t] >= t and ascending, so a
// tile's writes never reach the source of a later one.  A slot that is none is
// flagged where its row is moved.
__device__ __forceinline__ void move_weights(const PagedView &c, const EvictArgs &e, int row, int n) {
  constexpr int U = 16, TILE = U * MOVE_THREADS;
  const float *w = e.weights + row * e.w_stride;
  const int32_t *kept = e.kept + row * e.kept_stride;
  float *out = e.weights_out + row * e.w_out_stride;
  const uint32_t last = (static_cast<uint32_t>(c.max_pages) << c.page_shift) - 1;
  for (int base = 0; base < n; base += TILE) {
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = base + u * MOVE_THREADS + threadIdx.x;
      if (t < n) v[u] = w[min(static_cast<uint32_t>(kept[t]), last)];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = base + u * MOVE_THREADS + threadIdx.x;
      if (t < n) out[t] = v[u];
    }
  }
  for (int64_t t = n + threadIdx.x; t < e.w_out_stride; t += MOVE_THREADS) out[t] = 0.f;
}

// To other pages: every row on its own.  A CTA has COPY_ROWS rows of a
// (sequence, KV head): a thread first looks up one row's places (slot, page,
// destination: three dependent loads, once per row and not once per piece of
// it), then the K and V rows go over in 16-byte pieces, MOVE_ROWS of each in
// flight per thread.  `parts` CTAs for each head, and one more that moves the
// weights.
__global__ void __launch_bounds__(MOVE_THREADS) evict_copy_kernel(PagedView c, EvictArgs e, int parts) {
  __shared__ int64_t from[COPY_ROWS], to[COPY_ROWS];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int unit = blockIdx.x / (parts + 1), part = blockIdx.x % (parts + 1), b = unit / c.Hkv, g = unit % c.Hkv;
  const int n = min(paged_len(c, b, nullptr), e.keep);
  if (part == parts) {
    if (g == 0 && threadIdx.x == 0) e.new_lens[b] = n;
    if (g < e.Hs) move_weights(c, e, b * e.Hs + g, n);
    return;
  }
  const int base = part * COPY_ROWS, rows = min(n - base, COPY_ROWS);
  if (rows <= 0) return;
  const int32_t *kept = e.kept + (static_cast<int64_t>(b) * e.Hs + (e.Hs == 1 ? 0 : g)) * e.kept_stride + base;
  if (threadIdx.x < rows) {
    const int64_t f = src_offset(c, e, b, kept[threadIdx.x], g), t = dst_offset(c, e, b, base + threadIdx.x, g);
    from[threadIdx.x] = t < 0 ? -1 : f;
    to[threadIdx.x] = t;
  }
  __syncthreads();
  const int vecs = c.d / 8, per = MOVE_THREADS / vecs, x = threadIdx.x % vecs;
  for (int r0 = threadIdx.x / vecs; r0 < rows; r0 += per * MOVE_ROWS) {
    uint4 k[MOVE_ROWS], v[MOVE_ROWS];
#pragma unroll
    for (int u = 0; u < MOVE_ROWS; ++u) {
      const int r = r0 + u * per;
      if (r < rows && from[r] >= 0) {
        k[u] = reinterpret_cast<const uint4 *>(c.k + from[r])[x];
        v[u] = reinterpret_cast<const uint4 *>(c.v + from[r])[x];
      }
    }
#pragma unroll
    for (int u = 0; u < MOVE_ROWS; ++u) {
      const int r = r0 + u * per;
      if (r < rows && from[r] >= 0) {
        reinterpret_cast<uint4 *>(c.k + to[r])[x] = k[u];
        reinterpret_cast<uint4 *>(c.v + to[r])[x] = v[u];
      }
    }
  }
}

// In place: one CTA per (sequence, KV head), K or V and 64-byte slice of the
// rows walks the kept slots in order, a tile at a time; it reads the tile,
// waits for all its threads, and writes it.  kept[t] >= t and ascending, so a
// tile's writes never reach the source of a later tile; rows that stay where
// they are are skipped.  The slices give one sequence of 8 heads of 128 64
// CTAs.  The CTAs behind them move the weights.
constexpr int SHIFT_THREADS = 1024;

__global__ void __launch_bounds__(SHIFT_THREADS) evict_shift_kernel(PagedView c, EvictArgs e) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int parts = 2 * (c.d / 32);  // K or V, and the slice
  const int unit = blockIdx.x / parts, part = blockIdx.x % parts, b = unit / c.Hkv, g = unit % c.Hkv;
  const int n = min(paged_len(c, b, nullptr), e.keep);
  if (g == 0 && part == 0 && threadIdx.x == 0) e.new_lens[b] = n;
  __nv_bfloat16 *pages = part & 1 ? c.v : c.k;
  const int x = (part >> 1) * 4 + (threadIdx.x & 3), r = threadIdx.x >> 2;
  constexpr int per = SHIFT_THREADS / 4;
  const int32_t *kept = e.kept + (static_cast<int64_t>(b) * e.Hs + (e.Hs == 1 ? 0 : g)) * e.kept_stride;
  for (int base = 0; base < n; base += per * MOVE_ROWS) {
    int64_t to[MOVE_ROWS];
    uint4 v[MOVE_ROWS];
#pragma unroll
    for (int u = 0; u < MOVE_ROWS; ++u) {
      const int t = base + u * per + r, at = t < n ? kept[t] : t;
      to[u] = -1;
      if (at != t) {
        const int64_t from = src_offset(c, e, b, at, g);
        to[u] = from >= 0 ? dst_offset(c, e, b, t, g) : -1;
        if (to[u] >= 0) v[u] = reinterpret_cast<const uint4 *>(pages + from)[x];
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < MOVE_ROWS; ++u)
      if (to[u] >= 0) reinterpret_cast<uint4 *>(pages + to[u])[x] = v[u];
  }
}

__global__ void __launch_bounds__(MOVE_THREADS) evict_weights_kernel(PagedView c, EvictArgs e) {
  const int row = blockIdx.x;
  move_weights(c, e, row, min(paged_len(c, row / e.Hs, nullptr), e.keep));
}

// The frequencies of the last (d, theta) of this thread: 64 powers cost more
// than a small launch.
const RopeFreqs &rope_freqs(int d, double theta) {
  thread_local RopeFreqs f;
  thread_local int have_d = 0;
  thread_local double have_theta = 0.0;
  if (have_d != d || have_theta != theta) {
    fill_rope_freqs(&f, d, theta);
    have_d = d;
    have_theta = theta;
  }
  return f;
}

}  // namespace

spts_status launch_cache_append(const PagedView &c, const void *k_new, int64_t k_stride, const void *v_new,
                                int64_t v_stride, const int32_t *cu, int64_t T, const int32_t *pos, double theta,
                                uint32_t *status, cudaStream_t s) {
  if (T == 0) return SPTS_OK;
  const RopeFreqs &f = rope_freqs(c.d, theta);
  const int tokens = APPEND_THREADS / (c.d / 16);
  const unsigned blocks = static_cast<unsigned>((T + tokens - 1) / tokens);
  // Heads of a thread: 8 amortise the angles (32768 tokens of 8 heads: 49 us against 51 with 4 and 67 with 2), fewer
  // where that would leave SMs without a CTA.
  int heads = 8;
  while (heads > 1 && blocks * static_cast<unsigned>((c.Hkv + heads - 1) / heads) < static_cast<unsigned>(num_sms()))
    heads /= 2;
  const dim3 grid(blocks, static_cast<unsigned>((c.Hkv + heads - 1) / heads));
  const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(k_new), *v = static_cast<const __nv_bfloat16 *>(v_new);
  (c.d == 64 ? cache_append_kernel<64> : cache_append_kernel<128>)<<<grid, APPEND_THREADS, 0, s>>>(
      c, k, k_stride, v, v_stride, cu, static_cast<int>(T), pos, heads, f, status);
  note_launch();
  SPTS_CUDA_TRY(cudaGetLastError());
  return SPTS_OK;
}

spts_status launch_cache_evict(const PagedView &c, const EvictArgs &e, cudaStream_t s) {
  const int rows = c.B * e.Hs;
  const int64_t slots = static_cast<int64_t>(c.max_pages) << c.page_shift;
  const int64_t units = static_cast<int64_t>(c.B) * c.Hkv;
  const int64_t most = e.keep < slots ? e.keep : slots;
  const int parts = static_cast<int>((most + COPY_ROWS - 1) / COPY_ROWS);
  SPTS_REQUIRE(units * (parts + 1) < (int64_t(1) << 31), SPTS_ERR_SHAPE,
               "spts_cache_evict: too many rows for one call (%lld heads of sequences, %lld slots)",
               static_cast<long long>(units), static_cast<long long>(most));
  // CTAs per row: as many as there is an SM for, and enough to hold the keys
  int ctas = SEL_MAX_CLUSTER;
  while (ctas > 1 && rows * ctas > num_sms() && slots / (ctas / 2) <= SEL_MAX_KEYS - 32) ctas /= 2;
  const int64_t want = slots / ctas + 64;
  const int max_keys = static_cast<int>(want < SEL_MAX_KEYS ? want : SEL_MAX_KEYS);
  SPTS_TRY((allow_smem<evict_select_kernel>(SEL_MAX_KEYS * sizeof(uint32_t))));
  cudaLaunchAttribute cluster{};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = ctas;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * ctas);
  cfg.blockDim = dim3(SEL_THREADS);
  cfg.dynamicSmemBytes = max_keys * sizeof(uint32_t);
  cfg.stream = s;
  cfg.attrs = &cluster;
  cfg.numAttrs = 1;
  SPTS_CUDA_TRY(cudaLaunchKernelEx(&cfg, evict_select_kernel, c, e, ctas, max_keys));
  note_launch();
  if (e.dst_table == c.table) {
    SPTS_TRY(launch_behind(evict_shift_kernel, dim3(static_cast<unsigned>(units * 2 * (c.d / 32))), SHIFT_THREADS, s, 0,
                           c, e));
    evict_weights_kernel<<<rows, MOVE_THREADS, 0, s>>>(c, e);
    note_launch();
    SPTS_CUDA_TRY(cudaGetLastError());
    return SPTS_OK;
  }
  return launch_behind(evict_copy_kernel, dim3(static_cast<unsigned>(units * (parts + 1))), MOVE_THREADS, s, 0, c, e,
                       parts);
}

}  // namespace spts
