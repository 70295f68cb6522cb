// paged_weights.cu -- what each cached slot received from the new tokens of
// one attention call, added to its running weight:
//   weights[t] += sum over rows i and heads h of exp(scale q_ih . k_t - lse_ih)
//
// A second pass over K once the rows' lse are known: S is computed again,
// transposed, S^T = K Q^T, so that a TMEM lane is a slot and its sum over the
// rows stays inside one thread: no atomics, a fixed order, the same bits every
// time.  A unit is 256 slots (two K tiles of 128, one per warpgroup) of one KV
// head; it keeps its K tiles in shared memory while the Q tiles of the
// sequence (128 / G tokens x G heads each) stream past both, so Q comes from
// L2 once per 256 slots.  Bound by the exponentials (16384 per K and Q tile:
// 1024 cycles of the MUFU pipe against 256 of the MMA) when there are many
// rows, by reading K when there are few.  All exponentials are the MUFU
// pipe's: the output is fp32.
//   warp 0  TMA, warp 1  MMA, warps 4..7 and 8..11  slots of K tile 0 and 1
// With one weight row for all heads (Hs = 1) the units of a slot's KV heads
// leave partial sums that a last kernel adds in order, as long as their scratch
// stays below SPLIT_BYTES; beyond, a unit walks all its heads itself.
#include "host.hpp"
#include "paged.cuh"
#include "paged_plan.hpp"
#include "sm100.cuh"

namespace spts {
namespace {

constexpr int THREADS = 384;
constexpr int REG_LOW = 88, REG_HIGH = 208;  // 88 + 2 x 208 = 3 x 168
constexpr int BKV = PLAN_TILE;
constexpr int CHUNK = 128 * 64 * 2;
constexpr int MAX_SEQ = 1024;
constexpr uint32_t TMEM_COLS = 512;  // S of warpgroup x, buffer i: columns [256 x + 128 i, + 128)
constexpr float LOG2E = 1.4426950408889634f;
constexpr size_t SPLIT_BYTES = size_t(64) << 20;

struct Tail {
  int64_t before[MAX_SEQ + 1];  // units of the sequences before
  PlanSeq seq[MAX_SEQ];
  int first[MAX_SEQ];
  alignas(16) float2 lse[2][2][64];  // per warpgroup, by turns: -lse (log2) of the Q tile's rows, in pairs
  uint64_t q_full[2], q_empty[2], k_full[2], k_empty[2];
  uint64_t s_full[4], s_free[4], lse_full[4], drain;
  uint32_t tmem;
  int abort_flag;
};

struct Params {
  PagedView c;
  const int32_t *cu;
  int T, Hq, G, tq;
  int unit_heads;  // KV heads a unit walks: 1, or Hkv
  float scale_log2;
  const float *lse;
  float *out;  // row r = b * out_heads + (g or 0) at out + r * out_stride
  int out_heads;
  int64_t out_stride;
  int add;  // add to what is there (the weights), or write (partial sums)
  uint32_t *status;
  uint64_t wait_ns;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Unit {
  int b, g0, slot0;  // sequence, first KV head, first slot
  int q0, q1;        // Q tiles that see any of its slots
};

// Unit u of the list (sequence, pair of K tiles, head).
__device__ __forceinline__ Unit unit_at(const Tail &t, const Params &p, int64_t u) {
  int lo = 0, hi = p.c.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.before[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  const int per = p.c.Hkv / p.unit_heads;
  const int64_t i = u - t.before[lo];
  Unit r;
  r.b = lo;
  r.g0 = static_cast<int>(i % per) * p.unit_heads;
  r.slot0 = static_cast<int>(i / per) * 2 * BKV;
  const PlanSeq s = t.seq[lo];
  r.q0 = max(r.slot0 - (s.L - s.n), 0) / p.tq;  // the first token that sees slot0
  r.q1 = (s.n + p.tq - 1) / p.tq;
  return r;
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    paged_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ Params p) {
  constexpr int CH = D / 64, TILE = CH * CHUNK;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sQ = smem, *sK = smem + 2 * TILE;  // 2 Q tiles; 2 stages of 2 K tiles
  Tail &t = *reinterpret_cast<Tail *>(smem + 6 * TILE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int *abort_flag = &t.abort_flag;

  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) raise_status(p.status, SPTS_DEV_BADINDEX, 0x6Fu, smem_u32(smem));
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&t.q_full[i], 1);
      mbar_init(&t.q_empty[i], 1);
      mbar_init(&t.k_full[i], 1);
      mbar_init(&t.k_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&t.s_full[i], 1);
      mbar_init(&t.s_free[i], 4);  // one arrival per warp
      mbar_init(&t.lse_full[i], 4);
    }
    mbar_init(&t.drain, 1);
    t.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&t.tmem, TMEM_COLS);
    tmem_relinquish();
  }
  for (int b = threadIdx.x; b < p.c.B; b += THREADS) {
    int first, n;
    packed_span(p.cu, p.T, b, nullptr, first, n);
    t.first[b] = first;
    t.seq[b] = PlanSeq{n, paged_len(p.c, b, nullptr)};
  }
  __syncthreads();
  if (warp == 0) {
    int64_t run = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
      const int b = b0 + lane;
      int64_t x = 0;
      if (b < p.c.B && t.seq[b].n > 0)
        x = static_cast<int64_t>((t.seq[b].L + 2 * BKV - 1) / (2 * BKV)) * (p.c.Hkv / p.unit_heads);
      int64_t incl = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (b < p.c.B) t.before[b] = run + incl - x;
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) t.before[p.c.B] = run;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = t.tmem;
  const int64_t units = t.before[p.c.B];

  if (warp == 0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LOW));
    const int page = 1 << p.c.page_shift, rows = min(page, BKV), boxes = BKV / rows;
    const bool mine = lane < boxes * CH;
    const int box = lane / CH, ch = lane % CH;
    int qc = 0, kc = 0;
    uint32_t q_issued = 0, q_par = 0, k_issued = 0, k_par = 0;
    bool ok = true;
    auto wait_all = [&](uint64_t *bar, uint32_t parity, uint32_t where) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, p.wait_ns, where));
    };
    for (int64_t u = blockIdx.x; ok && u < units; u += gridDim.x) {
      const Unit un = unit_at(t, p, u);
      const int L = t.seq[un.b].L;
      int at[2];  // the pages of this lane's boxes, the same for every head; outside the tensor where there is none
      for (int x = 0; x < 2; ++x) {
        const int slot = un.slot0 + x * BKV + box * rows;
        at[x] = p.c.num_pages;
        if (mine && slot < L) {
          const int n = paged_page(p.c.table, p.c.table_stride, p.c.num_pages, un.b, slot >> p.c.page_shift, p.status);
          if (n >= 0) at[x] = n;
        }
      }
      if (un.q0 >= un.q1) continue;
      for (int h = 0; ok && h < p.unit_heads; ++h, ++kc) {
        const int g = un.g0 + h, st = kc & 1;
        const uint32_t ph = (kc >> 1) & 1;
        ok = wait_all(&t.k_empty[st], ph ^ 1u, 0x61u);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&t.k_full[st], 2 * TILE);
        __syncwarp();
        if (mine)
          for (int x = 0; x < 2; ++x)
            tma_load_4d(sK + (2 * st + x) * TILE + ch * CHUNK + box * rows * 128, &tmK, &t.k_full[st], ch * 64, g,
                        (un.slot0 + x * BKV) & (page - 1), at[x]);
        k_issued |= 1u << st;
        k_par = (k_par & ~(1u << st)) | (ph << st);
        for (int q = un.q0; q < un.q1; ++q, ++qc) {
          const int qs = qc & 1;
          const uint32_t qph = (qc >> 1) & 1;
          ok = wait_all(&t.q_empty[qs], qph ^ 1u, 0x62u);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&t.q_full[qs], p.tq * p.G * D * 2);
            for (int i = 0; i < CH; ++i)
              tma_load_3d(sQ + qs * TILE + i * CHUNK, &tmQ, &t.q_full[qs], i * 64, g * p.G,
                          t.first[un.b] + q * p.tq);
          }
          q_issued |= 1u << qs;
          q_par = (q_par & ~(1u << qs)) | (qph << qs);
        }
      }
    }
    if (*abort_flag && lane == 0)
      for (int i = 0; i < 2; ++i) {
        if (q_issued & (1u << i)) mbar_drain(&t.q_full[i], (q_par >> i) & 1u, p.status);
        if (k_issued & (1u << i)) mbar_drain(&t.k_full[i], (k_par >> i) & 1u, p.status);
      }
    __syncwarp();
  } else if (warp == 1) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LOW));
    constexpr uint32_t idesc = idesc_bf16_f32(BKV, 128, 0, 0);
    int qc = 0, kc = 0;
    bool ok = true;
    auto wait_all = [&](uint64_t *bar, uint32_t parity, uint32_t where) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, p.wait_ns, where));
    };
    for (int64_t u = blockIdx.x; ok && u < units; u += gridDim.x) {
      const Unit un = unit_at(t, p, u);
      if (un.q0 >= un.q1) continue;
      for (int h = 0; ok && h < p.unit_heads; ++h, ++kc) {
        const int st = kc & 1;
        ok = wait_all(&t.k_full[st], (kc >> 1) & 1, 0x63u);
        for (int q = un.q0; ok && q < un.q1; ++q, ++qc) {
          const int qs = qc & 1, buf = qc & 1;
          const uint32_t ph = (qc >> 1) & 1;
          ok = wait_all(&t.q_full[qs], ph, 0x64u);
          const uint32_t q_addr = smem_u32(sQ + qs * TILE);
          for (int x = 0; ok && x < 2; ++x) {
            ok = wait_all(&t.s_free[2 * x + buf], ph ^ 1u, 0x65u);
            if (!ok) break;
            tc_fence_after();
            const uint32_t k_addr = smem_u32(sK + (2 * st + x) * TILE);
#pragma unroll
            for (int kk = 0; kk < 4 * CH; ++kk) {
              const uint64_t a = sdesc_k_sw128(k_addr + (kk >> 2) * CHUNK) + 2 * (kk & 3);
              const uint64_t b = sdesc_k_sw128(q_addr + (kk >> 2) * CHUNK) + 2 * (kk & 3);
              mma_bf16_ss_w(tmem + x * 256 + buf * 128, a, b, idesc, kk > 0);
            }
            tc_commit_w(&t.s_full[2 * x + buf]);
          }
          if (ok) tc_commit_w(&t.q_empty[qs]);
        }
        if (ok) tc_commit_w(&t.k_empty[st]);
      }
    }
    tc_commit_w(&t.drain);
    mbar_drain(&t.drain, 0, p.status);
    __syncwarp();
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LOW));  // idle
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_HIGH));
    const int x = (warp - 4) >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16) + x * 256;
    const uint64_t cc = f2pack(p.scale_log2, p.scale_log2);
    const int rt = r / p.G, rh = r - rt * p.G;  // the token and head of Q row r (this thread fetches its lse)
    int qc = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; ok && u < units; u += gridDim.x) {
      const Unit un = unit_at(t, p, u);
      if (un.q0 >= un.q1) continue;
      const PlanSeq s = t.seq[un.b];
      const int slot = un.slot0 + x * BKV + r, base = s.L - s.n;
      uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
      for (int h = 0; ok && h < p.unit_heads; ++h) {
        const int head = (un.g0 + h) * p.G + rh;
        auto lse_of = [&](int q) -> float {
          const int tok = q * p.tq + rt;
          if (q >= un.q1 || rt >= p.tq || tok >= s.n) return 0.f;
          const float l = __ldg(p.lse + static_cast<int64_t>(t.first[un.b] + tok) * p.Hq + head);
          return l == -INFINITY ? 0.f : -LOG2E * l;  // a row that sees nothing: every column of it is masked
        };
        float next = lse_of(un.q0);
        for (int q = un.q0; q < un.q1; ++q, ++qc) {
          const int buf = qc & 1;
          const uint32_t ph = (qc >> 1) & 1;
          reinterpret_cast<float *>(t.lse[x][buf])[r] = next;
          mbar_arrive_warp(&t.lse_full[2 * x + buf]);
          next = lse_of(q + 1);
          ok = __all_sync(0xffffffffu, mbar_wait(&t.lse_full[2 * x + buf], ph, abort_flag, p.status, p.wait_ns, 0x66u));
          if (!ok) break;
          ok = __all_sync(0xffffffffu, mbar_wait(&t.s_full[2 * x + buf], ph, abort_flag, p.status, p.wait_ns, 0x67u));
          if (!ok) break;
          tc_fence_after();
          uint32_t xr[128];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            tmem_ld32(lane_base + buf * 128 + c * 32, *reinterpret_cast<uint32_t(*)[32]>(xr + 32 * c));
          tmem_ld_wait();
          tc_fence_before();
          mbar_arrive_warp(&t.s_free[2 * x + buf]);
          // rows of this tile that see the slot: tokens >= slot - base, up to the last one
          const int lo = (slot - base - q * p.tq) * p.G, hi = min(p.tq, s.n - q * p.tq) * p.G;
          if (__any_sync(0xffffffffu, lo > 0) || hi < 128) {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c < lo || c >= hi) xr[c] = 0xff800000u;  // -inf
          }
          const ulonglong2 *ls = reinterpret_cast<const ulonglong2 *>(t.lse[x][buf]);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const ulonglong2 l2 = ls[e];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int pair = 2 * e + i;
              const uint64_t a2 = f2fma(f2pack(__uint_as_float(xr[2 * pair]), __uint_as_float(xr[2 * pair + 1])), cc,
                                        i ? l2.y : l2.x);
              float a, b;
              if (pair % 5 == 1 || pair % 5 == 3) {  // two fifths on the FMA pipe
                exp2_fine2(a2, a, b);
              } else {
                f2unpack(a2, a, b);
                a = ex2(a);
                b = ex2(b);
              }
              sum[pair & 3] = f2add(sum[pair & 3], f2pack(a, b));
            }
          }
        }
      }
      if (!ok) break;
      if (slot < s.L) {
        float a, b, c, d;
        f2unpack(f2add(sum[0], sum[1]), a, b);
        f2unpack(f2add(sum[2], sum[3]), c, d);
        const float add = (a + b) + (c + d);
        float *w = p.out + (static_cast<int64_t>(un.b) * p.out_heads + (p.out_heads == 1 ? 0 : un.g0)) * p.out_stride + slot;
        *w = p.add ? *w + add : add;
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// weights[b, 0, t] += sum over g of part[b, g, t], t < L, for sequences with new tokens.
__global__ void __launch_bounds__(256) paged_weights_sum_kernel(PagedView c, const int32_t *cu, int T,
                                                                const float *__restrict__ part, int64_t part_stride,
                                                                float *__restrict__ w, int64_t w_stride) {
  const int b = blockIdx.y;
  int first, n;
  packed_span(cu, T, b, nullptr, first, n);
  const int L = paged_len(c, b, nullptr);
  if (n == 0) return;
  for (int64_t t = blockIdx.x * 256 + threadIdx.x; t < L; t += static_cast<int64_t>(gridDim.x) * 256) {
    float sum = 0.f;
    for (int g = 0; g < c.Hkv; ++g) sum += part[(static_cast<int64_t>(b) * c.Hkv + g) * part_stride + t];
    w[b * w_stride + t] += sum;
  }
}

// The same from the scores that the attention left (few rows): a thread has
// four slots and walks the rows that see them.  Bound by reading the scores
// and the weights.
__global__ void __launch_bounds__(128) stored_weights_kernel(PagedView c, const int32_t *__restrict__ cu, int T, int Hq,
                                                             float scale_log2, const float *scores,
                                                             int64_t score_stride, const float *lse, float *weights,
                                                             int Hs, int64_t w_stride, int chunks) {
  const int unit = blockIdx.x / chunks, chunk = blockIdx.x % chunks, b = unit / Hs, hs = unit % Hs;
  int first, n;
  packed_span(cu, T, b, nullptr, first, n);
  const int L = paged_len(c, b, nullptr), slot = (chunk * 128 + threadIdx.x) * 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (slot >= L || n == 0) return;
  const int heads = Hq / Hs, base = L - n;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = max(slot - base, 0); i < n; ++i) {
    const int64_t row = static_cast<int64_t>(first + i) * Hq + hs * heads;
    const int seen = base + i - slot;  // slots 0..seen of the four
#pragma unroll 4
    for (int h = 0; h < heads; ++h) {
      const float4 s = *reinterpret_cast<const float4 *>(scores + (row + h) * score_stride + slot);
      const float l = -LOG2E * lse[row + h];
      sum[0] += ex2(fmaf(s.x, scale_log2, l));
      if (seen >= 1) sum[1] += ex2(fmaf(s.y, scale_log2, l));
      if (seen >= 2) sum[2] += ex2(fmaf(s.z, scale_log2, l));
      if (seen >= 3) sum[3] += ex2(fmaf(s.w, scale_log2, l));
    }
  }
  float *w = weights + (static_cast<int64_t>(b) * Hs + hs) * w_stride + slot;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (slot + e < L) w[e] += sum[e];
}

template <int D>
spts_status launch(const CUtensorMap &q, const CUtensorMap &k, const Params &p, cudaStream_t s) {
  constexpr int bytes = 6 * (D / 64) * CHUNK + static_cast<int>(sizeof(Tail));
  SPTS_TRY((allow_smem<paged_weights_kernel<D>>(bytes)));
  paged_weights_kernel<D><<<num_sms(), THREADS, bytes, s>>>(q, k, p);
  note_launch();
  SPTS_CUDA_TRY(cudaGetLastError());
  return SPTS_OK;
}

}  // namespace

spts_status launch_stored_weights(const PagedView &c, const PagedAttnArgs &a, int64_t score_stride, cudaStream_t s) {
  const int64_t slots = static_cast<int64_t>(c.max_pages) << c.page_shift, chunks = (slots + 511) / 512;
  return launch_behind(stored_weights_kernel, dim3(static_cast<unsigned>(chunks * c.B * a.Hs)), 128, s, c, a.cu,
                       static_cast<int>(a.T), a.Hq, a.scale * LOG2E, static_cast<const float *>(a.scores), score_stride,
                       static_cast<const float *>(a.lse), a.weights, a.Hs, a.w_stride, static_cast<int>(chunks));
}

size_t paged_weights_scratch(int B, int64_t slots, int Hkv, int Hs) {
  const size_t n = static_cast<size_t>(B) * Hkv * slots;
  return Hs == 1 && Hkv > 1 && n * sizeof(float) <= SPLIT_BYTES ? n : 0;
}

spts_status launch_paged_weights(const PagedView &c, const PagedAttnArgs &a, const CUtensorMap &tmQ,
                                 const CUtensorMap &tmK, cudaStream_t s) {
  const int64_t slots = static_cast<int64_t>(c.max_pages) << c.page_shift;
  const bool split = paged_weights_scratch(c.B, slots, c.Hkv, a.Hs) > 0;
  Params p{};
  p.c = c;
  p.cu = a.cu;
  p.T = static_cast<int>(a.T);
  p.Hq = a.Hq;
  p.G = a.Hq / c.Hkv;
  p.tq = 128 / p.G;
  p.unit_heads = a.Hs == 1 && !split ? c.Hkv : 1;
  p.scale_log2 = a.scale * LOG2E;
  p.lse = a.lse;
  p.out = split ? a.w_scratch : a.weights;
  p.out_heads = split ? c.Hkv : a.Hs;
  p.out_stride = split ? slots : a.w_stride;
  p.add = split ? 0 : 1;
  p.status = a.status;
  p.wait_ns = wait_limit_ns();
  SPTS_TRY((c.d == 64 ? launch<64> : launch<128>)(tmQ, tmK, p, s));
  if (!split) return SPTS_OK;
  const unsigned blocks = static_cast<unsigned>((slots + 255) / 256);
  paged_weights_sum_kernel<<<dim3(blocks < 512 ? blocks : 512, c.B), 256, 0, s>>>(c, a.cu, p.T, a.w_scratch, slots,
                                                                                  a.weights, a.w_stride);
  note_launch();
  SPTS_CUDA_TRY(cudaGetLastError());
  return SPTS_OK;
}

}  // namespace spts
