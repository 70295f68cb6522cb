// api_paged.cu -- the extern "C" entry points of the paged key/value cache:
// host-side validation, workspace carving and dispatch.  See include/spts.h
// for the contract of every call.
#include <cmath>

#include "host.hpp"
#include "paged.cuh"

using namespace spts;

namespace {

inline cudaStream_t cs(spts_stream s) { return reinterpret_cast<cudaStream_t>(s); }

// Checks the descriptors and turns them into the kernels' view.
spts_status check_paged(const spts_attn_desc *a, const spts_paged_cache *c, const char *who, PagedView *view) {
  SPTS_REQUIRE(a != nullptr && c != nullptr, SPTS_ERR_INVALID, "%s: descriptor is NULL", who);
  SPTS_REQUIRE(a->dtype == SPTS_F32 || a->dtype == SPTS_BF16, SPTS_ERR_INVALID, "%s: unknown dtype", who);
  SPTS_REQUIRE(a->dtype == SPTS_BF16, SPTS_ERR_UNSUPPORTED, "%s: the paged cache is bf16", who);
  SPTS_REQUIRE(a->d == 64 || a->d == 128, SPTS_ERR_SHAPE, "%s: head dim must be 64 or 128 (d=%d)", who, a->d);
  SPTS_REQUIRE(a->Hq > 0 && a->Hkv > 0 && a->Hq % a->Hkv == 0, SPTS_ERR_SHAPE,
               "%s: need Hq, Hkv > 0 and Hq %% Hkv == 0 (Hq=%d Hkv=%d)", who, a->Hq, a->Hkv);
  SPTS_REQUIRE(a->Hq / a->Hkv <= 128, SPTS_ERR_UNSUPPORTED, "%s: need Hq / Hkv <= 128 (got %d)", who,
               a->Hq / a->Hkv);
  SPTS_REQUIRE(a->Hq <= (1 << 16), SPTS_ERR_SHAPE, "%s: too many heads (Hq=%d)", who, a->Hq);
  SPTS_REQUIRE(c->k_pages && c->v_pages && c->page_table && c->seq_lens, SPTS_ERR_INVALID, "%s: NULL argument", who);
  SPTS_REQUIRE(aligned(c->k_pages, 16) && aligned(c->v_pages, 16) && aligned(c->page_table, 4) &&
                   aligned(c->seq_lens, 4),
               SPTS_ERR_INVALID, "%s: misaligned pointer", who);
  const int S = c->page_size;
  SPTS_REQUIRE(S == 16 || S == 32 || S == 64 || S == 128 || S == 256, SPTS_ERR_UNSUPPORTED,
               "%s: page_size must be 16, 32, 64, 128 or 256 (got %d)", who, S);
  SPTS_REQUIRE(c->B >= 1 && c->B <= 1024, SPTS_ERR_SHAPE, "%s: need 1 <= B <= 1024 (B=%d)", who, c->B);
  SPTS_REQUIRE(c->num_pages >= 1 && c->num_pages < (int64_t(1) << 31) && c->max_pages >= 1 &&
                   static_cast<int64_t>(c->max_pages) * S <= (int64_t(1) << 30),
               SPTS_ERR_SHAPE, "%s: need num_pages >= 1 and 1 <= max_pages * page_size <= 2^30", who);
  const int64_t row = static_cast<int64_t>(a->Hkv) * a->d;
  const int64_t stride = c->page_stride ? c->page_stride : row * S;
  SPTS_REQUIRE(stride >= row * S && stride % 8 == 0 && stride < (int64_t(1) << 38), SPTS_ERR_SHAPE,
               "%s: page_stride must be a multiple of 8 and hold a page (%lld)", who, static_cast<long long>(stride));
  const int64_t ts = c->table_stride ? c->table_stride : c->max_pages;
  SPTS_REQUIRE(ts >= c->max_pages || c->B == 1, SPTS_ERR_SHAPE, "%s: table_stride below max_pages", who);
  int shift = 0;
  while ((1 << shift) < S) ++shift;
  *view = PagedView{static_cast<__nv_bfloat16 *>(c->k_pages),
                    static_cast<__nv_bfloat16 *>(c->v_pages),
                    c->page_table,
                    c->seq_lens,
                    stride,
                    ts,
                    static_cast<int>(c->num_pages),
                    shift,
                    c->B,
                    c->max_pages,
                    a->Hkv,
                    a->d};
  return SPTS_OK;
}

// A row stride of packed tokens: 0 means contiguous.
spts_status check_stride(int64_t *stride, int64_t row, const char *what, const char *who) {
  if (*stride == 0) *stride = row;
  SPTS_REQUIRE(*stride >= row && *stride % 8 == 0 && *stride < (int64_t(1) << 38), SPTS_ERR_SHAPE,
               "%s: %s must be a multiple of 8 and hold a row (%lld)", who, what, static_cast<long long>(*stride));
  return SPTS_OK;
}

// For either Hs, so that the workspace does not depend on it.
size_t weights_scratch(const spts_attn_desc *a, const spts_paged_cache *c) {
  return paged_weights_scratch(c->B, static_cast<int64_t>(c->max_pages) * c->page_size, a->Hkv, 1);
}

size_t attn_scratch(const spts_attn_desc *a, const spts_paged_cache *c, int64_t T) {
  return paged_attn_scratch_bytes(c->B, T, static_cast<int64_t>(c->max_pages) * c->page_size, a->Hq, a->Hkv, a->d);
}

size_t scores_bytes(const spts_attn_desc *a, const spts_paged_cache *c, int64_t T) {
  return paged_scores_bytes(c->B, T, static_cast<int64_t>(c->max_pages) * c->page_size, a->Hq, a->Hkv);
}

}  // namespace

extern "C" {

spts_status spts_cache_append(const spts_attn_desc *a, const spts_paged_cache *c, const void *k_new, int64_t k_stride,
                              const void *v_new, int64_t v_stride, const int32_t *cu_new, int64_t T,
                              const int32_t *pos, double theta, void *ws, spts_stream stream) {
  const char *who = "spts_cache_append";
  PagedView view;
  SPTS_TRY(check_paged(a, c, who, &view));
  SPTS_REQUIRE(T >= 0 && T < (int64_t(1) << 30), SPTS_ERR_SHAPE, "%s: need 0 <= T < 2^30 (T=%lld)", who,
               static_cast<long long>(T));
  SPTS_REQUIRE(cu_new && (T == 0 || (k_new && v_new)), SPTS_ERR_INVALID, "%s: NULL argument", who);
  SPTS_REQUIRE(aligned(k_new, 16) && aligned(v_new, 16) && aligned(cu_new, 4) && aligned(pos, 4), SPTS_ERR_INVALID,
               "%s: misaligned pointer", who);
  const int64_t row = static_cast<int64_t>(a->Hkv) * a->d;
  SPTS_TRY(check_stride(&k_stride, row, "k_stride", who));
  SPTS_TRY(check_stride(&v_stride, row, "v_stride", who));
  SPTS_REQUIRE(pos == nullptr || (std::isfinite(theta) && theta > 0.0), SPTS_ERR_INVALID, "%s: theta must be > 0",
               who);
  SPTS_REQUIRE(ws == nullptr || aligned(ws, 256), SPTS_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", who);
  return launch_cache_append(view, k_new, k_stride, v_new, v_stride, cu_new, T, pos, theta,
                             static_cast<uint32_t *>(ws), cs(stream));
}

size_t spts_paged_attention_workspace(const spts_attn_desc *a, const spts_paged_cache *c, int64_t T,
                                      int with_weights) {
  size_t b = kStatusBytes;
  if (a == nullptr || c == nullptr || T <= 0 || a->Hkv <= 0 || a->Hq < a->Hkv || a->Hq / a->Hkv > 128 || c->B <= 0 ||
      c->max_pages <= 0 || c->page_size <= 0)
    return b;
  b += Carver::round(attn_scratch(a, c, T));
  if (with_weights) {
    b += Carver::round(static_cast<size_t>(T) * a->Hq * sizeof(float));  // lse
    const size_t scores = scores_bytes(a, c, T);
    b += Carver::round(scores ? scores : weights_scratch(a, c) * sizeof(float));
  }
  return b;
}

spts_status spts_paged_attention(const spts_attn_desc *a, const spts_paged_cache *c, const void *q, int64_t q_stride,
                                 const int32_t *cu_q, int64_t T, void *o, int64_t o_stride, float *lse,
                                 float *weights, int Hs, int64_t w_stride, void *ws, size_t ws_bytes,
                                 spts_stream stream) {
  const char *who = "spts_paged_attention";
  PagedView view;
  SPTS_TRY(check_paged(a, c, who, &view));
  SPTS_REQUIRE(T >= 0 && T < (int64_t(1) << 30), SPTS_ERR_SHAPE, "%s: need 0 <= T < 2^30 (T=%lld)", who,
               static_cast<long long>(T));
  SPTS_REQUIRE(cu_q && (T == 0 || (q && o)), SPTS_ERR_INVALID, "%s: NULL argument", who);
  SPTS_REQUIRE(aligned(q, 16) && aligned(o, 16) && aligned(cu_q, 4) && aligned(lse, 4) && aligned(weights, 4),
               SPTS_ERR_INVALID, "%s: misaligned pointer", who);
  SPTS_REQUIRE(T == 0 || o != q, SPTS_ERR_INVALID, "%s: o must not alias q", who);
  const int64_t row = static_cast<int64_t>(a->Hq) * a->d;
  SPTS_TRY(check_stride(&q_stride, row, "q_stride", who));
  SPTS_TRY(check_stride(&o_stride, row, "o_stride", who));
  if (weights) {
    SPTS_REQUIRE(Hs == 1 || Hs == a->Hkv, SPTS_ERR_SHAPE, "%s: Hs must be 1 or Hkv (Hs=%d)", who, Hs);
    SPTS_REQUIRE(w_stride >= static_cast<int64_t>(c->max_pages) * c->page_size, SPTS_ERR_SHAPE,
                 "%s: w_stride below max_pages * page_size (%lld)", who, static_cast<long long>(w_stride));
  }
  SPTS_TRY(check_ws(ws, ws_bytes, spts_paged_attention_workspace(a, c, T, weights != nullptr), who));
  if (T == 0) return SPTS_OK;
  Carver cv(ws, ws_bytes);
  PagedAttnArgs args{q, q_stride, cu_q, T, a->Hq, 0.f, o, o_stride, lse, weights, weights ? Hs : 1, w_stride,
                     cv.status(), cv.take(attn_scratch(a, c, T)), nullptr, nullptr};
  args.scale = a->scale > 0.f ? a->scale : 1.0f / std::sqrt(static_cast<float>(a->d));
  if (weights) {
    float *own = static_cast<float *>(cv.take(static_cast<size_t>(T) * a->Hq * sizeof(float)));
    if (lse == nullptr) args.lse = own;
    const size_t scores = scores_bytes(a, c, T);
    float *rest = static_cast<float *>(cv.take(scores ? scores : weights_scratch(a, c) * sizeof(float)));
    (scores ? args.scores : args.w_scratch) = rest;
  }
  return launch_paged_attention(view, args, cs(stream));
}

size_t spts_cache_evict_workspace(const spts_paged_cache *c, int Hs, int64_t keep) {
  if (c == nullptr || Hs <= 0 || keep <= 0 || c->B <= 0 || c->max_pages <= 0) return kStatusBytes;
  const int64_t cap = static_cast<int64_t>(c->max_pages) * c->page_size;
  return kStatusBytes + Carver::round(static_cast<size_t>(c->B) * Hs * (keep < cap ? keep : cap) * sizeof(int32_t));
}

spts_status spts_cache_evict(const spts_attn_desc *a, const spts_paged_cache *c, const float *weights, int Hs,
                             int64_t w_stride, int64_t keep, int64_t sink, int64_t recent, const int32_t *dst_table,
                             int dst_max_pages, int64_t dst_stride, float *weights_out, int64_t w_out_stride,
                             int32_t *new_lens, int32_t *kept_idx, void *ws, size_t ws_bytes, spts_stream stream) {
  const char *who = "spts_cache_evict";
  PagedView view;
  SPTS_TRY(check_paged(a, c, who, &view));
  SPTS_REQUIRE(weights && dst_table && weights_out && new_lens, SPTS_ERR_INVALID, "%s: NULL argument", who);
  SPTS_REQUIRE(aligned(weights, 4) && aligned(dst_table, 4) && aligned(weights_out, 4) && aligned(new_lens, 4) &&
                   aligned(kept_idx, 4),
               SPTS_ERR_INVALID, "%s: misaligned pointer", who);
  SPTS_REQUIRE(Hs == 1 || Hs == a->Hkv, SPTS_ERR_SHAPE, "%s: Hs must be 1 or Hkv (Hs=%d)", who, Hs);
  SPTS_REQUIRE(keep >= 1 && keep < (int64_t(1) << 31) && sink >= 0 && recent >= 0 && sink <= keep &&
                   recent <= keep - sink,
               SPTS_ERR_SHAPE, "%s: need keep >= 1, sink, recent >= 0 and sink + recent <= keep (%lld, %lld, %lld)",
               who, static_cast<long long>(keep), static_cast<long long>(sink), static_cast<long long>(recent));
  const int64_t cap = static_cast<int64_t>(c->max_pages) * c->page_size;
  const int64_t most = keep < cap ? keep : cap;
  SPTS_REQUIRE(w_stride >= cap, SPTS_ERR_SHAPE, "%s: w_stride below max_pages * page_size (%lld)", who,
               static_cast<long long>(w_stride));
  SPTS_REQUIRE(w_out_stride >= most && w_out_stride < (int64_t(1) << 31), SPTS_ERR_SHAPE,
               "%s: w_out_stride below min(keep, max_pages * page_size) (%lld)", who,
               static_cast<long long>(w_out_stride));
  SPTS_REQUIRE(weights != weights_out || w_stride == w_out_stride, SPTS_ERR_SHAPE,
               "%s: weights_out is weights, but the strides differ", who);
  if (dst_stride == 0) dst_stride = dst_max_pages;
  SPTS_REQUIRE(dst_max_pages >= 1 && (dst_stride >= dst_max_pages || c->B == 1), SPTS_ERR_SHAPE,
               "%s: need dst_max_pages >= 1 and dst_stride >= dst_max_pages", who);
  SPTS_REQUIRE(dst_table != c->page_table || dst_stride == view.table_stride || c->B == 1, SPTS_ERR_SHAPE,
               "%s: dst_table is page_table, but the strides differ", who);
  SPTS_TRY(check_ws(ws, ws_bytes, spts_cache_evict_workspace(c, Hs, keep), who));
  Carver cv(ws, ws_bytes);
  int32_t *kept = static_cast<int32_t *>(cv.take(static_cast<size_t>(c->B) * Hs * most * sizeof(int32_t)));
  EvictArgs e{weights,
              Hs,
              w_stride,
              static_cast<int>(keep),
              static_cast<int>(sink),
              static_cast<int>(recent),
              dst_table,
              dst_max_pages,
              dst_stride,
              weights_out,
              w_out_stride,
              new_lens,
              kept_idx ? kept_idx : kept,
              kept_idx ? keep : most,
              cv.status()};
  return launch_cache_evict(view, e, cs(stream));
}

}  // extern "C"
