// paged_attn.cu -- attention of new tokens over the paged cache.
#include "host.hpp"
#include "paged.cuh"

namespace spts {
namespace {

// Sequence and place of packed row t.
struct Row {
  int b, i, n, L;
};

__device__ __forceinline__ bool row_of(const PagedView &c, const int32_t *cu, int T, int t, uint32_t *status, Row &r) {
  if (t >= __ldg(cu + c.B)) return false;
  int lo = 0, hi = c.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  int first;
  packed_span(cu, T, lo, status, first, r.n);
  r.b = lo;
  r.i = t - first;
  r.L = paged_len(c, lo, status);
  return r.i >= 0 && r.i < r.n;
}

// One warp per (row, query head): each lane holds d / 32 columns, one pass
// over the visible slots with the running maximum and sum.
template <int D>
__global__ void __launch_bounds__(128) paged_attn_rows_kernel(PagedView c, PagedAttnArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int t = static_cast<int>(unit / a.Hq), h = static_cast<int>(unit % a.Hq), g = h / (a.Hq / c.Hkv);
  Row r;
  if (blockIdx.x == 0) check_sequences(c, a.cu, static_cast<int>(a.T), a.status);
  if (t >= a.T || !row_of(c, a.cu, static_cast<int>(a.T), t, nullptr, r)) return;
  const int end = max(r.L - r.n + r.i + 1, 0);
  float q[E], acc[E], m = -INFINITY, l = 0.f;
  const __nv_bfloat16 *qr = static_cast<const __nv_bfloat16 *>(a.q) + t * a.q_stride + h * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(qr[e]) * a.scale;
    acc[e] = 0.f;
  }
  int page = -1;
  for (int j = 0; j < end; ++j) {
    if ((j & ((1 << c.page_shift) - 1)) == 0)
      page = paged_page(c.table, c.table_stride, c.num_pages, r.b, j >> c.page_shift, lane == 0 ? a.status : nullptr);
    if (page < 0) continue;
    const int64_t at = paged_offset(c, page, j, g) + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], __bfloat162float(c.k[at + e]), s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mn = fmaxf(m, s);
    const float top = mn == -INFINITY ? 0.f : mn;  // no score above -inf yet (a NaN keeps its p NaN)
    const float f = m == -INFINITY ? 0.f : expf(m - mn), p = expf(s - top);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(p, __bfloat162float(c.v[at + e]), acc[e] * f);
    m = mn;
  }
  __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + t * a.o_stride + h * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = __float2bfloat16(l == 0.f ? 0.f : acc[e] / l);
  if (lane == 0 && a.lse) a.lse[static_cast<int64_t>(t) * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

// One thread per (sequence, weight row, slot): the weights of every new row
// and head over again, from the rows' lse.
template <int D>
__global__ void __launch_bounds__(128) paged_weights_kernel(PagedView c, PagedAttnArgs a) {
  const int b = blockIdx.y / a.Hs, hs = blockIdx.y % a.Hs, j = blockIdx.x * 128 + threadIdx.x;
  int first, n;
  packed_span(a.cu, static_cast<int>(a.T), b, nullptr, first, n);
  const int L = paged_len(c, b, nullptr);
  if (j >= L || n == 0) return;
  const int page = paged_page(c.table, c.table_stride, c.num_pages, b, j >> c.page_shift, a.status);
  if (page < 0) return;
  const int heads = a.Hq / a.Hs, G = a.Hq / c.Hkv;
  float sum = 0.f;
  for (int i = max(0, j - (L - n)); i < n; ++i)
    for (int h = hs * heads; h < (hs + 1) * heads; ++h) {
      const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + (first + i) * a.q_stride + h * D;
      const __nv_bfloat16 *k = c.k + paged_offset(c, page, j, h / G);
      float s = 0.f;
      for (int e = 0; e < D; ++e) s = fmaf(__bfloat162float(q[e]) * a.scale, __bfloat162float(k[e]), s);
      sum += expf(s - a.lse[static_cast<int64_t>(first + i) * a.Hq + h]);
    }
  a.weights[(static_cast<int64_t>(b) * a.Hs + hs) * a.w_stride + j] += sum;
}

}  // namespace

spts_status launch_paged_attention(const PagedView &c, const PagedAttnArgs &a, cudaStream_t s) {
  if (a.T == 0) return SPTS_OK;
  const unsigned blocks = static_cast<unsigned>((a.T * a.Hq + 3) / 4);
  if (c.d == 64) paged_attn_rows_kernel<64><<<blocks, 128, 0, s>>>(c, a);
  else paged_attn_rows_kernel<128><<<blocks, 128, 0, s>>>(c, a);
  note_launch();
  SPTS_CUDA_TRY(cudaGetLastError());
  if (a.weights == nullptr) return SPTS_OK;
  const int cap = c.max_pages << c.page_shift;
  const dim3 grid(static_cast<unsigned>((cap + 127) / 128), static_cast<unsigned>(c.B) * a.Hs);
  if (c.d == 64) paged_weights_kernel<64><<<grid, 128, 0, s>>>(c, a);
  else paged_weights_kernel<128><<<grid, 128, 0, s>>>(c, a);
  note_launch();
  SPTS_CUDA_TRY(cudaGetLastError());
  return SPTS_OK;
}

}  // namespace spts
