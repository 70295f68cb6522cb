// paged_weights.cu -- what each cached slot received from the new tokens of
// one attention call, added to its running weight:
//   weights[t] += sum over rows i and heads h of exp(scale q_ih . k_t - lse_ih)
//
// A second pass over K once the rows' lse are known: S is computed again,
// transposed, S^T = K Q^T, so that a TMEM lane is a slot and its sum over the
// rows stays inside one thread: no atomics, a fixed order, the same bits every
// time.  A unit is up to four K tiles of 128 slots of one KV head, one for each
// of four warpgroups; they stay in shared memory while the Q tiles of the
// sequence (128 / G tokens x G heads each) stream past all four.  (With two K
// tiles per Q tile the Q loads were what everything waited for: without any
// exponential 250 rows over 32K slots still took 90 of 126 us.)  With one or
// two K tiles the warpgroups share out the Q tiles instead, and their sums are
// added in order at the end: 7
// sequences of 685 new tokens in 738, 2 heads of 8 (84 K tiles), 68 -> 46 us.
// The sums over the Q tiles keep what they round away (LongSum): with 8 x 4 heads
// a prompt of 8192 rows adds 2048 tiles to a slot's weight over all heads.
// Bound by the
// exponentials (16384 per K and Q tile: 1024 cycles of the MUFU pipe against
// 512 of the MMA) when there are many rows, by reading K when there are few.
// All exponentials are the MUFU pipe's: the output is fp32.
//   warp 0  TMA, warp 1  MMA, warp 3  hands out the units, warps 4..19  four
//   warpgroups, one per K tile
// The K tiles of all sequences and heads, weighted with the Q tiles that see
// them, are shared out evenly; a CTA's share is cut into units at heads and
// fours.
// With one weight row for all heads (Hs = 1) the units of a slot's KV heads
// leave partial sums that a last kernel adds in order, as long as their scratch
// stays below SPLIT_BYTES; beyond, a unit walks all its heads itself.
#include "host.hpp"
#include "paged.cuh"
#include "paged_plan.hpp"
#include "sm100.cuh"

namespace spts {
namespace {

constexpr int THREADS = 640;
constexpr int REG_LOW = 56, REG_HIGH = 104;  // 56 + 4 x 104 <= 5 x 96, the launch allocation
constexpr int WG = 4;  // warpgroups, and K tiles of a unit at most
constexpr int ROUNDS = 4;    // K tiles of a CTA, at most, that are dealt out one by one
constexpr int LISTED = 640;  // and in all
constexpr int LISTED_STEPS = 9;  // from so many Q tiles per K tile on
constexpr int BKV = PLAN_TILE;
constexpr int CHUNK = 128 * 64 * 2;
constexpr int MAX_SEQ = 1024;
constexpr uint32_t TMEM_COLS = 512;  // S^T of warpgroup w: columns [128 w, 128 w + 128)
constexpr float LOG2E = 1.4426950408889634f;
constexpr size_t SPLIT_BYTES = size_t(64) << 20;

constexpr int ITEMS = 4;

// A unit, as the warps need it.
struct Unit {
  int more;          // 0 behind the last
  int b, n, L;       // the sequence, its new and cached tokens
  int first;         // packed row of its first new token
  int g0, slot0;     // first KV head, first slot
  int tiles;         // K tiles
  int share;         // warpgroups that share a K tile's Q tiles
  int q0, q1;        // Q tiles that see any of its slots
};

struct Tail {
  int64_t before[MAX_SEQ + 1];  // cost of the sequences before, all heads (few K tiles: how many)
  PlanSeq seq[MAX_SEQ];
  int first[MAX_SEQ];
  alignas(16) float lse[WG][2][128];  // per warpgroup, by turns: -lse (log2) of the Q tile's rows
  uint64_t q_full[2], q_empty[2], k_full[WG], k_empty[WG];
  float join[WG][128];  // the sums of a warpgroup that shares the K tile of another one
  uint64_t s_full[WG], s_free[WG], lse_full[2 * WG], join_full[WG], join_free[WG], drain;
  uint64_t item_full[ITEMS], item_empty[ITEMS];
  Unit item[ITEMS];
  uint32_t tmem;
  int listed;        // all K tiles, where they are dealt out one by one; otherwise 0
  int mine[ROUNDS];  // then: this CTA's, or -1
  alignas(16) int cost[LISTED];
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

// A sum of many parts that keeps what each addition rounds away (Kahan 1965): as
// good as one rounding, however many.  Added one by one in fp32, 16384 weights of
// 0.1 are off by 1.5e-4 of their sum, and small ones behind large ones are lost.
struct LongSum {
  float sum, lost;
  __device__ __forceinline__ void add(float part) {
    const float y = part - lost, s = sum + y;
    lost = (s - sum) - y;
    sum = s;
  }
};

__device__ __forceinline__ int k_tiles(int L) { return (L + BKV - 1) / BKV; }

// K tile i of a call with few of them.
struct KeyTile {
  int b, g, j;
};
__device__ __forceinline__ KeyTile key_tile(const Tail &t, const Params &p, int i) {
  int lo = 0, hi = p.c.B;
  while (lo < hi) {  // the first sequence that ends behind it
    const int mid = (lo + hi) >> 1;
    if (t.before[mid + 1] <= i) lo = mid + 1;
    else hi = mid;
  }
  const int in = i - static_cast<int>(t.before[lo]), tiles = k_tiles(t.seq[lo].L);
  return KeyTile{lo, in / tiles, in % tiles};
}

// Few K tiles, whose costs differ: an equal share of the cost would end in the
// middle of most of them (148 alike, a few cheaper, on 148 CTAs: 332 us, and 210
// one by one).  In the order of falling cost they go round the CTAs, to and fro.
// With fewer than LISTED_STEPS Q tiles per K tile, units of several K tiles save
// more (480 K tiles, us with the attention: 1 Q tile each 47 one by one, 35 in
// shares; 8: 92, 89; 10 to 15: 49, 52 and 102, 112).  All threads.
__device__ __forceinline__ void deal_out(Tail &t, const Params &p) {
  const int total = t.listed, ctas = gridDim.x, x = blockIdx.x;
  for (int i = threadIdx.x; i < LISTED; i += THREADS) {
    int cost = 0;
    if (i < total) {
      const KeyTile k = key_tile(t, p, i);
      cost = static_cast<int>(plan_keys_cost(t.seq[k.b], p.tq, k.j + 1) - plan_keys_cost(t.seq[k.b], p.tq, k.j));
    }
    t.cost[i] = cost;
  }
  if (threadIdx.x < ROUNDS) t.mine[threadIdx.x] = -1;
  __syncthreads();
  const int i = threadIdx.x;
  if (i < total) {
    const int4 *cost = reinterpret_cast<const int4 *>(t.cost);
    const int own = t.cost[i];
    int rank = 0;  // tiles in front of this one
    for (int k = 0; k < total; k += 4) {
      const int4 c = cost[k >> 2];
      rank += (c.x + (k < i) > own) + (c.y + (k + 1 < i) > own) + (c.z + (k + 2 < i) > own) + (c.w + (k + 3 < i) > own);
    }
    const int round = rank / ctas, at = rank - round * ctas;
    if (x == (round & 1 ? ctas - 1 - at : at)) t.mine[round] = i;
  }
  __syncthreads();
}

// Warp 3, one lane: this CTA's units, handed to the other warps through a
// ring.  K tiles are ordered by (sequence, head, slot); a tile belongs to the
// CTA whose equal share of the cost its first position falls into.
__device__ __forceinline__ void walk(Tail &t, const Params &p) {
  volatile int *abort_flag = &t.abort_flag;
  const int heads = p.c.Hkv / p.unit_heads;  // head by head, or all at once
  const int64_t total = t.before[p.c.B];
  const int64_t lo = plan_cut(total, gridDim.x, blockIdx.x), hi = plan_cut(total, gridDim.x, blockIdx.x + 1);
  int count = 0;
  auto place = [&]() -> Unit * {
    const int i = count % ITEMS;
    const bool ok =
        mbar_wait_long(&t.item_empty[i], ((count / ITEMS) & 1) ^ 1, abort_flag, p.status, p.wait_ns, 0x60u);
    return ok ? &t.item[i] : nullptr;
  };
  // `take` K tiles of a head from tile j on; false: the kernel is on its way out
  auto hand_out = [&](int b, int g, int j, int take) -> bool {
    Unit *r = place();
    if (r == nullptr) return false;
    const PlanSeq s = t.seq[b];
    r->more = 1;
    r->b = b;
    r->n = s.n;
    r->L = s.L;
    r->first = t.first[b];
    r->g0 = g * p.unit_heads;
    r->slot0 = j * BKV;
    r->tiles = take;
    r->q0 = max(j * BKV - (s.L - s.n), 0) / p.tq;  // the first token that sees the first slot
    r->q1 = plan_windows(s.n, p.tq);               // > q0: the last token sees every slot below L
    r->share = plan_sharers(take, r->q1 - r->q0);
    mbar_arrive(&t.item_full[count % ITEMS]);
    ++count;
    return true;
  };
  if (t.listed) {
    for (int i = 0; i < ROUNDS && t.mine[i] >= 0; ++i) {
      const KeyTile k = key_tile(t, p, t.mine[i]);
      if (!hand_out(k.b, k.g, k.j, 1)) return;
    }
  }
  int b0 = t.listed ? p.c.B : 0;
  for (int end = p.c.B; b0 < end;) {  // the first sequence that ends behind lo
    const int mid = (b0 + end) >> 1;
    if (t.before[mid + 1] <= lo) b0 = mid + 1;
    else end = mid;
  }
  for (int b = b0; b < p.c.B && t.before[b] < hi; ++b) {
    const PlanSeq s = t.seq[b];
    const int tiles = k_tiles(s.L);
    if (tiles == 0 || s.n == 0) continue;
    // tiles [from, to) of the sequence's tiles of all heads begin in this share
    const int64_t head = plan_keys_cost(s, p.tq, tiles);
    auto index_at = [&](int64_t x) -> int64_t {
      if (x <= 0) return 0;
      const int64_t g = plan_div(x, head);
      return g >= heads ? static_cast<int64_t>(heads) * tiles : g * tiles + plan_keys_at(s, p.tq, tiles, x - g * head);
    };
    const int64_t from = index_at(lo - t.before[b]), to = index_at(hi - t.before[b]);
    int g = static_cast<int>(from / tiles), j = static_cast<int>(from - static_cast<int64_t>(g) * tiles);
    for (int64_t k = from; k < to;) {
      const int64_t left = to - k;
      const int take = min(tiles - j, left < WG ? static_cast<int>(left) : WG);
      if (!hand_out(b, g, j, take)) return;
      k += take;
      j += take;
      if (j == tiles) {
        j = 0;
        ++g;
      }
    }
  }
  Unit *r = place();
  if (r == nullptr) return;
  r->more = 0;
  mbar_arrive(&t.item_full[count % ITEMS]);
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    paged_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ Params p) {
  constexpr int CH = D / 64, TILE = CH * CHUNK;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sQ = smem, *sK = smem + 2 * TILE;  // a ring of 2 Q tiles; one of K tiles
  Tail &t = *reinterpret_cast<Tail *>(smem + 6 * TILE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int *abort_flag = &t.abort_flag;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) raise_status(p.status, SPTS_DEV_BADINDEX, 0x6Fu, smem_u32(smem));
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&t.q_full[i], 1);
      mbar_init(&t.q_empty[i], 1);
    }
    for (int i = 0; i < WG; ++i) {
      mbar_init(&t.k_full[i], 1);
      mbar_init(&t.k_empty[i], 1);
      mbar_init(&t.s_full[i], 1);
      mbar_init(&t.s_free[i], 4);  // here and below: one arrival per warp
      mbar_init(&t.lse_full[2 * i], 4);
      mbar_init(&t.lse_full[2 * i + 1], 4);
      mbar_init(&t.join_full[i], 4);
      mbar_init(&t.join_free[i], 4);
    }
    for (int i = 0; i < ITEMS; ++i) {
      mbar_init(&t.item_full[i], 1);
      mbar_init(&t.item_empty[i], 18);  // a lane of every other warp that takes part
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
    const int heads = p.c.Hkv / p.unit_heads;
    int64_t run = 0, k_total = 0, steps = 0;  // all K tiles; the Q tiles that they are multiplied with, at most
    for (int b = lane; b < p.c.B; b += 32)
      if (t.seq[b].n > 0) {
        const int64_t tiles = static_cast<int64_t>(k_tiles(t.seq[b].L)) * heads;
        k_total += tiles;
        steps += tiles * plan_windows(t.seq[b].n, p.tq);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      k_total += __shfl_xor_sync(0xffffffffu, k_total, o);
      steps += __shfl_xor_sync(0xffffffffu, steps, o);
    }
    const bool few = k_total <= ROUNDS * static_cast<int64_t>(gridDim.x) && k_total <= LISTED &&
                     steps >= LISTED_STEPS * k_total;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
      const int b = b0 + lane;
      int64_t x = 0;
      if (b < p.c.B && t.seq[b].n > 0) {
        const int tiles = k_tiles(t.seq[b].L);
        x = (few ? tiles : plan_keys_cost(t.seq[b], p.tq, tiles)) * heads;
      }
      int64_t incl = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (b < p.c.B) t.before[b] = run + incl - x;
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      t.before[p.c.B] = run;
      t.listed = few ? static_cast<int>(k_total) : 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (t.listed) deal_out(t, p);
  const uint32_t tmem = uniform(t.tmem);
  // launched while the attention still runs: nothing that it writes (lse, the
  // scratch) is touched before this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // The i-th unit for this warp, or null behind the last one (or on the way
  // out); give_back lets warp 3 reuse its place.
  auto take = [&](int i) -> const Unit * {
    const bool ok = __all_sync(0xffffffffu, mbar_wait_long(&t.item_full[i % ITEMS], (i / ITEMS) & 1, abort_flag,
                                                           p.status, p.wait_ns, 0x6Fu));
    const Unit *un = &t.item[i % ITEMS];
    return ok && uniform(un->more) ? un : nullptr;
  };
  auto give_back = [&](int i) { mbar_arrive_warp(&t.item_empty[i % ITEMS]); };

  if (warp == 0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LOW));
    const int page = 1 << p.c.page_shift, rows = min(page, BKV), boxes = BKV / rows;
    const bool mine = lane < boxes * CH;
    const int box = lane / CH, ch = lane % CH;
    int qs = 0, k0 = 0;  // where the next Q and K tiles go
    uint32_t qph = 0;
    uint32_t q_issued = 0, q_par = 0, k_issued = 0, k_par = 0;  // k_par: the parity of each K place's next phase
    bool ok = true;
    auto wait_all = [&](uint64_t *bar, uint32_t parity, uint32_t where) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, p.wait_ns, where));
    };
    for (int i = 0; ok; ++i) {
      const Unit *un = take(i);
      if (!un) break;
      const int L = un->L, g0 = un->g0, q0 = uniform(un->q0), q1 = uniform(un->q1), slot0 = un->slot0, b = un->b;
      const int first = un->first, tiles = uniform(un->tiles);
      give_back(i);
      int at[WG];  // the pages of this lane's boxes, the same for every head; outside the tensor where there is none
#pragma unroll
      for (int w = 0; w < WG; ++w) {
        const int slot = slot0 + w * BKV + box * rows;
        at[w] = p.c.num_pages;
        if (mine && w < tiles && slot < L) {
          const int n = paged_page(p.c.table, p.c.table_stride, p.c.num_pages, b, slot >> p.c.page_shift, p.status);
          if (n >= 0) at[w] = n;
        }
      }
      for (int h = 0; ok && h < p.unit_heads; ++h) {
        const int g = g0 + h;
#pragma unroll
        for (int w = 0; w < WG; ++w) {
          if (w >= tiles || !ok) break;
          const int x = (k0 + w) & (WG - 1);
          ok = wait_all(&t.k_empty[x], ((k_par >> x) & 1u) ^ 1u, 0x61u);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&t.k_full[x], TILE);
          __syncwarp();
          if (mine)
            tma_load_4d(sK + x * TILE + ch * CHUNK + box * rows * 128, &tmK, &t.k_full[x], ch * 64, g,
                        (slot0 + w * BKV) & (page - 1), at[w]);
          k_issued |= 1u << x;
          k_par ^= 1u << x;
        }
        k0 = (k0 + tiles) & (WG - 1);
        for (int q = q0; ok && q < q1; ++q) {
          ok = wait_all(&t.q_empty[qs], qph ^ 1u, 0x62u);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&t.q_full[qs], p.tq * p.G * D * 2);
            for (int e = 0; e < CH; ++e)
              tma_load_3d(sQ + qs * TILE + e * CHUNK, &tmQ, &t.q_full[qs], e * 64, g * p.G, first + q * p.tq);
          }
          q_issued |= 1u << qs;
          q_par = (q_par & ~(1u << qs)) | (qph << qs);
          qs ^= 1;
          qph ^= qs ^ 1;
        }
      }
    }
    if (*abort_flag && lane == 0) {
      for (int i = 0; i < 2; ++i)
        if (q_issued & (1u << i)) mbar_drain(&t.q_full[i], (q_par >> i) & 1u, p.status);
      for (int i = 0; i < WG; ++i)
        if (k_issued & (1u << i)) mbar_drain(&t.k_full[i], ((k_par >> i) & 1u) ^ 1u, p.status);
    }
    __syncwarp();
  } else if (warp == 1) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LOW));
    constexpr uint32_t idesc = idesc_bf16_f32(BKV, 128, 0, 0);
    int qs = 0, k0 = 0;
    uint32_t qph = 0, k_par = 0, s_par = 0;  // parity of the next load of each K place, of the next S of each warpgroup
    bool ok = true;
    auto wait_all = [&](uint64_t *bar, uint32_t parity, uint32_t where) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, p.wait_ns, where));
    };
    for (int i = 0; ok; ++i) {
      const Unit *un = take(i);
      if (!un) break;
      const int n = uniform(un->q1 - un->q0), tiles = uniform(un->tiles), share = uniform(un->share);
      give_back(i);
      for (int h = 0; ok && h < p.unit_heads; ++h) {
        int x = 0;  // first warpgroup of this Q tile
        for (int q = 0; ok && q < n; ++q) {
          ok = wait_all(&t.q_full[qs], qph, 0x64u);
          const uint32_t q_addr = smem_u32(sQ + qs * TILE);
          for (int w = 0; ok && w < tiles; ++w) {
            const int kw = (k0 + w) & (WG - 1), wg = x + w;
            if (q == 0) ok = wait_all(&t.k_full[kw], (k_par >> kw) & 1u, 0x63u);
            ok = ok && wait_all(&t.s_free[wg], ((s_par >> wg) & 1u) ^ 1u, 0x65u);
            if (!ok) break;
            s_par ^= 1u << wg;
            tc_fence_after();
            const uint32_t k_addr = smem_u32(sK + kw * TILE);
#pragma unroll
            for (int kk = 0; kk < 4 * CH; ++kk) {
              const uint64_t a = sdesc_k_sw128(k_addr + (kk >> 2) * CHUNK) + 2 * (kk & 3);
              const uint64_t b = sdesc_k_sw128(q_addr + (kk >> 2) * CHUNK) + 2 * (kk & 3);
              mma_bf16_ss_w(tmem + wg * 128, a, b, idesc, kk > 0);
            }
            tc_commit_w(&t.s_full[wg]);
            if (q + 1 == n) tc_commit_w(&t.k_empty[kw]);
          }
          if (ok) tc_commit_w(&t.q_empty[qs]);
          x = x + tiles == share * tiles ? 0 : x + tiles;
          qs ^= 1;
          qph ^= qs ^ 1;
        }
        for (int w = 0; w < tiles; ++w) k_par ^= 1u << ((k0 + w) & (WG - 1));
        k0 = (k0 + tiles) & (WG - 1);
      }
    }
    tc_commit_w(&t.drain);
    mbar_drain(&t.drain, 0, p.status);
    __syncwarp();
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LOW));
    if (warp == 3 && lane == 0) walk(t, p);  // warp 2 is idle
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_HIGH));
    const int wg = (warp - 4) >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16) + wg * 128;
    const float c2 = p.scale_log2;
    const int rt = r / p.G, rh = r - rt * p.G;  // token and head of Q row r, whose lse this thread fetches
    uint32_t sc = 0;                            // S tiles of this warpgroup so far
    uint32_t join_par = 0;                      // per warpgroup: parity of its next sums for another one
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const Unit *un = take(i);
      if (!un) break;
      const int tiles = uniform(un->tiles), share = uniform(un->share), part = wg / tiles;
      const int n = un->n, L = un->L, q0 = un->q0 + part, q1 = un->q1, g0 = un->g0, first = un->first;
      const int slot = un->slot0 + (wg - part * tiles) * BKV + r, base = L - n;
      const int64_t out_row = static_cast<int64_t>(un->b) * p.out_heads + (p.out_heads == 1 ? 0 : g0);
      float *w = p.out + out_row * p.out_stride + slot;
      give_back(i);
      const uint32_t joined = join_par;
      join_par ^= ((1u << (share * tiles)) - 1u) & ~((1u << tiles) - 1u);
      if (part >= share) continue;
      const float old = p.add && part == 0 && slot < L ? *w : 0.f;
      // lse of this thread's row of Q tile q, fetched a tile ahead
      auto lse_of = [&](int h, int q) -> float {
        const int tok = q * p.tq + rt;
        if (rt >= p.tq || tok >= n) return 0.f;
        const float l = __ldg(p.lse + static_cast<int64_t>(first + tok) * p.Hq + (g0 + h) * p.G + rh);
        return l == -INFINITY ? 0.f : -LOG2E * l;  // a row that sees nothing: every column of it is masked
      };
      float next = lse_of(0, q0);
      LongSum tiles_sum{};  // over the Q tiles; inside one, four sums of 32
      for (int h = 0; ok && h < p.unit_heads; ++h) {
        for (int q = q0; q < q1; q += share, ++sc) {
          uint64_t *lse_full = &t.lse_full[2 * wg + (sc & 1)];
          t.lse[wg][sc & 1][r] = next;
          mbar_arrive_warp(lse_full);
          next = q + share < q1 ? lse_of(h, q + share) : h + 1 < p.unit_heads ? lse_of(h + 1, q0) : 0.f;
          ok = __all_sync(0xffffffffu, mbar_wait(lse_full, (sc >> 1) & 1, abort_flag, p.status, p.wait_ns, 0x66u));
          if (!ok) break;
          ok = __all_sync(0xffffffffu, mbar_wait(&t.s_full[wg], sc & 1, abort_flag, p.status, p.wait_ns, 0x67u));
          if (!ok) break;
          tc_fence_after();
          // rows of the tile that see the slot: tokens >= slot - base, up to the last one
          const int lo = (slot - base - q * p.tq) * p.G, hi = min(p.tq, n - q * p.tq) * p.G;
          const bool early = __any_sync(0xffffffffu, lo > 0);  // some slot of this warp is behind some row
          const float4 *ls = reinterpret_cast<const float4 *>(t.lse[wg][sc & 1]);
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t xr[64];
#pragma unroll
            for (int c = 0; c < 2; ++c)
              tmem_ld32(lane_base + half * 64 + c * 32, *reinterpret_cast<uint32_t(*)[32]>(xr + 32 * c));
            tmem_ld_wait();
            if (half) {
              tc_fence_before();
              mbar_arrive_warp(&t.s_free[wg]);
            }
            if (early) {
              if (__all_sync(0xffffffffu, lo >= half * 64 + 64)) continue;  // no slot of this warp is seen
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (half * 64 + c < lo) xr[c] = 0xff800000u;  // -inf
            }
            if (hi < half * 64 + 64) {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (half * 64 + c >= hi) xr[c] = 0xff800000u;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float4 l4 = ls[half * 16 + e];
              sum[0] += ex2(fmaf(__uint_as_float(xr[4 * e]), c2, l4.x));
              sum[1] += ex2(fmaf(__uint_as_float(xr[4 * e + 1]), c2, l4.y));
              sum[2] += ex2(fmaf(__uint_as_float(xr[4 * e + 2]), c2, l4.z));
              sum[3] += ex2(fmaf(__uint_as_float(xr[4 * e + 3]), c2, l4.w));
            }
          }
          tiles_sum.add((sum[0] + sum[1]) + (sum[2] + sum[3]));
        }
      }
      if (!ok) break;
      float total = tiles_sum.sum;
      if (part > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&t.join_free[wg], ((joined >> wg) & 1u) ^ 1u, abort_flag, p.status,
                                               p.wait_ns, 0x68u));
        if (!ok) break;
        t.join[wg][r] = total;
        mbar_arrive_warp(&t.join_full[wg]);
        continue;
      }
      for (int x = wg + tiles; ok && x < share * tiles; x += tiles) {
        ok = __all_sync(0xffffffffu, mbar_wait(&t.join_full[x], (joined >> x) & 1u, abort_flag, p.status, p.wait_ns,
                                               0x69u));
        if (!ok) break;
        total += t.join[x][r];
        mbar_arrive_warp(&t.join_free[x]);
      }
      if (!ok) break;
      if (slot < L) *w = old + total;
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
                                                                const float *part, int64_t part_stride, float *w,
                                                                int64_t w_stride) {
  const int b = blockIdx.y;
  int first, n;
  packed_span(cu, T, b, nullptr, first, n);
  const int L = paged_len(c, b, nullptr);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (n == 0) return;
  for (int64_t t = blockIdx.x * 256 + threadIdx.x; t < L; t += static_cast<int64_t>(gridDim.x) * 256) {
    float sum = 0.f;
    for (int g = 0; g < c.Hkv; ++g) sum += part[(static_cast<int64_t>(b) * c.Hkv + g) * part_stride + t];
    w[b * w_stride + t] += sum;
  }
}

// The same from the scores that the attention left (few rows).  A lane has
// four slots, a CTA's warps take turns with the rows, and their sums are added
// in order.  Bound by reading the scores and the weights; the turns shorten
// the chain of loads where a slot has many rows (up to 20 rows of 4 heads over
// 438 slots: the whole call 28 us against 43).
constexpr int STORED_WARPS = 4;
// More weights than this of a warp go to long sums, block by block (always doing so took registers: 16 rows of 8 x 4
// heads, the whole call 70.9 us against 70.0; 69.4 without any).
constexpr int STORED_BLOCK = 32;

__global__ void __launch_bounds__(32 * STORED_WARPS)
    stored_weights_kernel(PagedView c, const int32_t *__restrict__ cu, int T, int Hq, float scale_log2,
                          const float *scores, int64_t score_stride, const float *lse, float *weights, int Hs,
                          int64_t w_stride, int chunks) {
  __shared__ float4 sums[STORED_WARPS][32];
  const int unit = blockIdx.x / chunks, chunk = blockIdx.x % chunks, b = unit / Hs, hs = unit % Hs;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int first, n;
  packed_span(cu, T, b, nullptr, first, n);
  const int L = paged_len(c, b, nullptr), slot = (chunk * 32 + lane) * 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (chunk * 128 >= L || n == 0) return;
  const int heads = Hq / Hs, base = L - n;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  int i = warp / heads, h = warp % heads;  // row and head
  int e = warp;
  auto add_rows = [&](int end) {
#pragma unroll 4
    for (; e < end; e += STORED_WARPS) {
      const int64_t row = static_cast<int64_t>(first + i) * Hq + hs * heads + h;
      const int seen = base + i - slot;  // the row sees slots 0..seen of the four
      if (slot < L && seen >= 0) {
        const float4 s = *reinterpret_cast<const float4 *>(scores + row * score_stride + slot);
        const float l = -LOG2E * lse[row];
        sum[0] += ex2(fmaf(s.x, scale_log2, l));
        if (seen >= 1) sum[1] += ex2(fmaf(s.y, scale_log2, l));
        if (seen >= 2) sum[2] += ex2(fmaf(s.z, scale_log2, l));
        if (seen >= 3) sum[3] += ex2(fmaf(s.w, scale_log2, l));
      }
      h += STORED_WARPS;
      while (h >= heads) {
        h -= heads;
        ++i;
      }
    }
  };
  const int rows = n * heads;
  if (rows <= STORED_BLOCK * STORED_WARPS) {
    add_rows(rows);
  } else {
    LongSum total[4]{};
    while (e < rows) {
      add_rows(min(rows, e + STORED_BLOCK * STORED_WARPS));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        total[k].add(sum[k]);
        sum[k] = 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k] = total[k].sum;
  }
  sums[warp][lane] = make_float4(sum[0], sum[1], sum[2], sum[3]);
  __syncthreads();
  // thread t adds up and writes slot t of the 128
  const int t = threadIdx.x, at = chunk * 128 + t;
  float add = 0.f;
#pragma unroll
  for (int q = 0; q < STORED_WARPS; ++q) add += reinterpret_cast<const float *>(sums[q])[t];
  if (at < L) weights[(static_cast<int64_t>(b) * Hs + hs) * w_stride + at] += add;
}

template <int D>
spts_status launch(const CUtensorMap &q, const CUtensorMap &k, const Params &p, cudaStream_t s) {
  constexpr int bytes = 6 * (D / 64) * CHUNK + static_cast<int>(sizeof(Tail));
  SPTS_TRY((allow_smem<paged_weights_kernel<D>>(bytes)));
  return launch_behind(paged_weights_kernel<D>, dim3(num_sms()), THREADS, s, bytes, q, k, p);
}

}  // namespace

spts_status launch_stored_weights(const PagedView &c, const PagedAttnArgs &a, int64_t score_stride, cudaStream_t s) {
  const int64_t slots = static_cast<int64_t>(c.max_pages) << c.page_shift, chunks = (slots + 127) / 128;
  const dim3 grid(static_cast<unsigned>(chunks * c.B * a.Hs));
  return launch_behind(stored_weights_kernel, grid, 32 * STORED_WARPS, s, 0, c, a.cu,
                       static_cast<int>(a.T), a.Hq, a.scale * LOG2E, static_cast<const float *>(a.scores), score_stride,
                       static_cast<const float *>(a.lse), a.weights, a.Hs, a.w_stride, static_cast<int>(chunks));
}

size_t paged_weights_scratch(int B, int64_t slots, int Hkv, int Hs) {
  const size_t n = static_cast<size_t>(B) * Hkv * slots;
  return Hs == 1 && Hkv > 1 && n * sizeof(float) <= SPLIT_BYTES ? n : 0;
}

spts_status launch_paged_weights(const PagedView &c, const PagedAttnArgs &a, const CUtensorMap &tmK, cudaStream_t s) {
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
  CUtensorMap tmQ;
  SPTS_TRY(paged_q_map(c, a, p.tq, &tmQ));
  SPTS_TRY((c.d == 64 ? launch<64> : launch<128>)(tmQ, tmK, p, s));
  if (!split) return SPTS_OK;
  const unsigned blocks = static_cast<unsigned>((slots + 255) / 256);
  return launch_behind(paged_weights_sum_kernel, dim3(blocks < 512 ? blocks : 512, c.B), 256, s, 0, c, a.cu, p.T,
                       static_cast<const float *>(a.w_scratch), slots, a.weights, a.w_stride);
}

}  // namespace spts
