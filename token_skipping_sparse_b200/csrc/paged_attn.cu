// paged_attn.cu -- attention of new tokens over the paged cache, on tcgen05.
//
// For query row (token i of a sequence, head h) and the slots t it sees,
//   s_t = scale q . k_t,   o = sum_t 2^(s_t' - m) v_t / l,   l = sum_t 2^(s_t' - m)
// with s' = s log2(e) and m the running maximum: one pass over the keys.
//
// A Q tile packs tq = 128 / G tokens x the G query heads of one KV head into
// the 128 rows of an MMA; a unit is two such tiles (a window of 2 tq tokens)
// and one KV head.  Bound by the tensor pipe and the exponentials when the
// windows are full, by reading K and V once when there are few new tokens:
// then a unit's rows are the same but most of them are padding, and what
// counts is that K and V stream without a pause.  So one persistent CTA per
// SM takes an equal share of all units' key slots, wherever the cuts fall
// (paged_plan.hpp): one request over 128K slots and 64 requests of ragged
// lengths both load every SM alike.  Units that a cut divides leave partial
// results (unnormalised O, m, l) that the combine kernel joins, in order.
//   warp 0      TMA: Q tiles, and K and V tiles of 128 slots into two rings;
//               a tile is gathered from its pages, one box per page and 64
//               columns, each issued by a lane of its own.  Pages past the
//               sequence's last one (and bad page numbers) are loaded from
//               outside the tensor: zeros;
//   warp 1      MMA: S_x = Q_x K^T into TMEM, then O_x += P_x V with P_x read
//               from TMEM; the loop runs across units without a drain;
//   warp 2      zeroes the V rows behind the sequence's last slot in its last
//               tile (they may hold anything, and 0 x NaN is NaN), between
//               that tile's load and the MMA warp;
//   warp 3      walks the plan and hands the pieces to the other warps through
//               a ring of ITEMS places, ahead of them;
//   warps 4..7, 8..11  softmax, one thread per row, one warpgroup per S_x.
// A unit with two tiles gives them to x = 0 and 1, and every K/V tile feeds
// both.  A unit with one (n <= tq: decoding) gives the even key tiles to x = 0
// and the odd ones to x = 1, with the same Q, and joins the two at the end:
// the softmax of one key tile runs beside the MMAs of the next either way.
// P is rounded to bf16 for the product with V (half a step: 2^-8 of each
// weight at most); S, the maxima, the sums and O stay in fp32.
// All barrier waits are bounded (see sm100.cuh).
#include <type_traits>

#include "host.hpp"
#include "paged.cuh"
#include "paged_plan.hpp"
#include "sm100.cuh"

namespace spts {
namespace {

constexpr int THREADS = 384;
// setmaxnreg split: each SMSP holds one warp of warpgroup 0 and one softmax
// warp of each tile: 88 + 2 x 208 = 3 x 168, the launch allocation.
constexpr int REG_LOW = 88, REG_HIGH = 208;
constexpr int BKV = PLAN_TILE;
constexpr int CHUNK = 128 * 64 * 2;   // 128 rows of 64 bf16, 128-byte swizzle
constexpr int MAX_SEQ = 1024;
constexpr uint32_t TMEM_COLS = 512;   // S_0 [0,128), S_1 [128,256), O_0 from 256, O_1 from 384
constexpr float RESCALE_THRESHOLD = 8.0f;  // log2 units
constexpr float LN2 = 0.69314718055994530942f;
// One column pair in POLY_EVERY takes its exp2 from the FMA pipe (exp2_poly2,
// 1e-4, far below P's bf16 step) when the row sums serve the bf16 output
// alone.  Where lse or weights are wanted all are the MUFU pipe's: a degree-5
// polynomial (2.6e-7) for two fifths of them cost more registers than it gave
// (250 rows over 32K slots: 141 us against 134).
constexpr int POLY_EVERY = 3;

// Which units a launch is made for.  FULL: windows of two full Q tiles.  FEW:
// the same, and an extra path for units of at most 16 rows (without it the
// full units' loop is a little faster: an 8K prompt 480 us against 499).
// STEP: windows of one Q tile of at most 16 rows; its place in shared memory
// goes to a third stage of K and V, and one warp per S_x is the softmax (64
// ragged sequences: 211 us against 224 with FEW).
enum Mode { FULL, FEW, STEP };

template <int D, Mode MODE>
struct Geometry {
  static constexpr int CH = D / 64;                 // 64-column chunks of a row
  static constexpr int TILE = CH * CHUNK;           // a Q, K or V tile
  static constexpr int STAGES = (MODE == STEP ? 3 : 2) * (D == 128 ? 1 : 2);  // of K and of V
  // With STEP only 16 rows of a Q tile are there; the MMA reads 128 from its
  // place on, and the rows of S behind the first 16 are not looked at.
  static constexpr int Q_CHUNK = MODE == STEP ? 16 * 128 : CHUNK;
  static constexpr int Q_TILE = CH * Q_CHUNK;
  static constexpr int WARPS = MODE == STEP ? 1 : 4;  // softmax warps per S_x
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 2 * Q_TILE;
  static constexpr int OFF_V = OFF_K + STAGES * TILE;
  static constexpr int OFF_TAIL = OFF_V + STAGES * TILE;
};

constexpr int ITEMS = 4;

// A piece of a unit, as the warps need it.
struct Item {
  int more;           // 0 behind the last piece
  int b, n, L;        // the sequence, its new and cached tokens
  int first;          // packed row of its first new token
  int tok0;           // first token of the window
  int g;              // KV head
  int two;            // whether the window fills a second Q tile
  int t0, t1;         // key tiles
  int a_end;          // with two Q tiles: end of those that the first one goes over
  int whole;          // the piece is the unit
  int part;           // otherwise: place of its partial result
};

struct Tail {  // shared memory behind the tiles
  int64_t before[MAX_SEQ + 1];
  PlanSeq seq[MAX_SEQ];
  int first[MAX_SEQ];
  float2 xchg[2][2][128];  // by turns: a warpgroup without a tile may be one piece ahead
  uint64_t q_full[2], q_empty[2], k_full[6], k_empty[6], v_full[6], v_empty[6];
  uint64_t v_raw[6];  // instead of v_full where a tile's V goes through warp 2
  uint64_t s_full[2], p_ready[4], o_done[2], o_free, x_full, drain;
  uint64_t item_full[ITEMS], item_empty[ITEMS];
  Item item[ITEMS];
  uint32_t tmem;
  int abort_flag;
  int groups, group_heads;  // KV heads are taken in `groups` groups of at most group_heads
};

template <int D, Mode MODE>
constexpr size_t smem_bytes() {
  constexpr size_t bytes = Geometry<D, MODE>::OFF_TAIL + sizeof(Tail);
  static_assert(bytes <= 232448, "more shared memory than a CTA can have");
  return bytes;
}

struct Params {
  PagedView c;
  const int32_t *cu;
  int T, Hq, G;
  int tq, w;        // tokens of a Q tile and of a window
  int slot_rows;    // rows of a partial result: w G, rounded up
  int whole;        // units are dealt out whole
  int max_groups;   // head groups that the scratch has room for
  float scale_log2;
  __nv_bfloat16 *o;
  int64_t o_stride;
  float *lse;
  float *part_o;    // [max_groups][ctas][2][slot_rows][D]
  float2 *part_ml;  // [max_groups][ctas][2][slot_rows]: running maximum (log2) and sum
  PlanCut *cuts;    // [max_groups][ctas]
  float *scores;    // [T, Hq, score_stride] or NULL: q . k of every row and slot, for the weights
  int64_t score_stride;
  uint32_t *status;
  uint64_t wait_ns;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Maxima that keep a NaN: a row that sees one comes out as NaN.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 32 bytes at once: a row's thread writes whole sectors.
__device__ __forceinline__ void store_8(float *to, const float *v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// TMEM in rows of 16: thread t of the warp has row t / 4 (and t / 4 + 8) and,
// of every 8 fp32 columns, columns 2 (t % 4) and the next.  ld: 8 N columns, 4 N
// values {row, row, row + 8, row + 8}; st: 4 N columns of bf16 pairs, 2 N values
// {row, row + 8}, so the pair a thread has loaded goes to the column it is at.
__device__ __forceinline__ void tmem_ld_rows16(uint32_t addr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]),
        "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]),
        "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
        "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
        "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_rows16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ PlanShape shape_of(const Params &p) { return PlanShape{p.w, p.tq}; }
__device__ __forceinline__ int heads_of(const Tail &t, const Params &p, int group) {
  return max(min(t.group_heads, p.c.Hkv - group * t.group_heads), 0);
}

// Warp 3, one lane: the pieces of this CTA's ranges, group after group, or
// every gridDim.x-th unit.
__device__ __forceinline__ void walk(Tail &t, const Params &p) {
  volatile int *abort_flag = &t.abort_flag;
  const int w = p.w, r = blockIdx.x;
  int count = 0;
  auto place = [&]() -> Item * {  // the next free place of the ring
    const int i = count % ITEMS;
    const bool ok =
        mbar_wait_long(&t.item_empty[i], ((count / ITEMS) & 1) ^ 1, abort_flag, p.status, p.wait_ns, 0x50u);
    return ok ? &t.item[i] : nullptr;
  };
  auto hand_out = [&](const PlanPiece &pc, int g, int part) -> bool {
    Item *it = place();
    if (it == nullptr) return false;
    const PlanSeq s = t.seq[pc.b];
    it->more = 1;
    it->b = pc.b;
    it->n = s.n;
    it->L = s.L;
    it->first = t.first[pc.b];
    it->tok0 = pc.p * w;
    it->g = g;
    it->two = w > p.tq && s.n - pc.p * w > p.tq;
    it->t0 = pc.t0;
    it->t1 = pc.t1;
    it->a_end = plan_first_end(s, shape_of(p), pc.p, pc.t0, pc.t1);
    it->whole = pc.whole;
    it->part = part;
    mbar_arrive(&t.item_full[count % ITEMS]);
    ++count;
    return true;
  };
  if (p.whole) {
    PlanPiece pc{};
    pc.whole = 1;
    const int64_t units = t.before[p.c.B] * p.c.Hkv;
    for (int64_t u = r; u < units; u += gridDim.x) {
      while (t.before[pc.b + 1] * p.c.Hkv <= u) ++pc.b;
      const int64_t i = u - t.before[pc.b] * p.c.Hkv;
      pc.p = static_cast<int>(plan_div(i, p.c.Hkv));
      pc.t1 = (plan_visible(t.seq[pc.b], (pc.p + 1) * w) + BKV - 1) / BKV;
      if (!hand_out(pc, static_cast<int>(i - static_cast<int64_t>(pc.p) * p.c.Hkv), 0)) return;
    }
  } else {
    for (int group = 0; group < t.groups; ++group) {
      const int heads = heads_of(t, p, group);
      const int64_t total = t.before[p.c.B] * heads;
      const int nr = plan_ranges(total, gridDim.x);
      if (r >= nr) continue;
      const int64_t x = plan_cut(total, nr, r);
      PlanCursor cur;
      plan_open(cur, t.seq, t.before, p.c.B, shape_of(p), heads, x, plan_cut(total, nr, r + 1) - x);
      PlanPiece pc;
      while (plan_next(cur, t.seq, p.c.B, shape_of(p), heads, pc)) {
        if (pc.t0 >= pc.t1 && !pc.whole) continue;  // nothing to compute, nothing to write
        if (!hand_out(pc, group * t.group_heads + pc.g, (group * static_cast<int>(gridDim.x) + r) * 2 + pc.slot))
          return;
      }
    }
  }
  Item *it = place();
  if (it == nullptr) return;
  it->more = 0;
  mbar_arrive(&t.item_full[count % ITEMS]);
}

// Lengths and offsets of all sequences, and their costs added up.
__device__ __forceinline__ void read_sequences(Tail &t, const Params &p) {
  uint32_t *status = blockIdx.x == 0 ? p.status : nullptr;
  for (int b = threadIdx.x; b < p.c.B; b += THREADS) {
    int first, n;
    packed_span(p.cu, p.T, b, status, first, n);
    t.first[b] = first;
    t.seq[b] = PlanSeq{n, paged_len(p.c, b, status)};
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int64_t run = 0, shared = 0;  // cost; slots of sequences with several windows
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
      const int b = b0 + lane;
      int64_t x = 0;
      if (b < p.c.B && t.seq[b].n > p.w) shared += t.seq[b].L;
      if (b < p.c.B && p.whole) x = plan_windows(t.seq[b].n, p.w);
      else if (b < p.c.B) x = plan_cost(plan_base(t.seq[b], shape_of(p)), plan_windows(t.seq[b].n, p.w), p.w);
      int64_t incl = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (b < p.c.B) t.before[b] = run + incl - x;
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) shared += __shfl_xor_sync(0xffffffffu, shared, o);
    if (lane == 0) {
      t.before[p.c.B] = run;
      t.groups = plan_groups(shared * p.c.Hkv * p.c.d * 4, run * p.c.Hkv, gridDim.x, p.c.Hkv, p.max_groups);
      t.group_heads = (p.c.Hkv + t.groups - 1) / t.groups;
    }
  }
  __syncthreads();
}

template <int D, bool EXACT, Mode MODE>
__global__ void __launch_bounds__(THREADS, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  using Gm = Geometry<D, MODE>;
  constexpr int CH = Gm::CH, TILE = Gm::TILE, STAGES = Gm::STAGES, WARPS = Gm::WARPS;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sQ = smem + Gm::OFF_Q, *sK = smem + Gm::OFF_K, *sV = smem + Gm::OFF_V;
  Tail &t = *reinterpret_cast<Tail *>(smem + Gm::OFF_TAIL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int *abort_flag = &t.abort_flag;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) raise_status(p.status, SPTS_DEV_BADINDEX, 0x5Fu, smem_u32(smem));
    return;
  }
  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&t.q_full[x], 1);
      mbar_init(&t.q_empty[x], 1);
      mbar_init(&t.s_full[x], 1);
      mbar_init(&t.p_ready[2 * x], WARPS);  // here and below: one arrival per warp
      mbar_init(&t.p_ready[2 * x + 1], WARPS);
      mbar_init(&t.o_done[x], 1);
    }
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&t.k_full[s], 1);
      mbar_init(&t.k_empty[s], 1);
      mbar_init(&t.v_full[s], 1);
      mbar_init(&t.v_empty[s], 1);
      mbar_init(&t.v_raw[s], 1);
    }
    mbar_init(&t.o_free, 2 * WARPS);
    mbar_init(&t.x_full, 2 * WARPS);
    for (int i = 0; i < ITEMS; ++i) {
      mbar_init(&t.item_full[i], 1);
      mbar_init(&t.item_empty[i], 3 + 2 * WARPS);  // warps 0 to 2 and the softmax
    }
    mbar_init(&t.drain, 1);
    t.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&t.tmem, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  read_sequences(t, p);  // ends with __syncthreads
  tc_fence_after();
  const uint32_t tmem = uniform(t.tmem);
  // The i-th item for this warp, or null behind the last one (or on the way
  // out); give_back lets warp 3 reuse its place.
  auto take = [&](int i) -> const Item * {
    const bool ok = __all_sync(0xffffffffu, mbar_wait_long(&t.item_full[i % ITEMS], (i / ITEMS) & 1, abort_flag,
                                                           p.status, p.wait_ns, 0x5Fu));
    const Item *it = &t.item[i % ITEMS];
    return ok && uniform(it->more) ? it : nullptr;
  };
  auto give_back = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&t.item_empty[i % ITEMS]);
  };

  if (warp == 0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LOW));
    // ---------------- TMA, the whole warp: lane l issues box l of a tile
    const int page = 1 << p.c.page_shift, rows = min(page, BKV), boxes = BKV / rows;
    const bool mine = lane < boxes * CH;
    const int box = lane / CH, ch = lane % CH;
    int qc = 0, kc = 0;  // Q tiles and K/V tiles loaded so far
    uint32_t k_issued = 0, k_par = 0, v_issued = 0, v_par = 0, v_raw = 0, raw_par = 0, q_issued = 0, q_par = 0;
    bool ok = true;
    auto wait_all = [&](uint64_t *bar, uint32_t parity, uint32_t where) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, p.wait_ns, where));
    };
    // the page of this lane's box in tile j; outside the tensor where there is none
    auto page_of = [&](int b, int L, int j) -> int {
      const int slot = j * BKV + box * rows;
      if (!mine || slot >= L) return p.c.num_pages;
      const int n = paged_page(p.c.table, p.c.table_stride, p.c.num_pages, b, slot >> p.c.page_shift, p.status);
      return n < 0 ? p.c.num_pages : n;
    };
    for (int i = 0; ok; ++i) {
      const Item *it = take(i);
      if (!it) break;
      const int b = it->b, t0 = uniform(it->t0), t1 = uniform(it->t1), g = it->g, L = it->L;
      const int row0 = it->first + it->tok0, tiles_q = uniform(it->two) ? 2 : 1;
      give_back(i);
      int next = t0 < t1 ? page_of(b, L, t0) : 0;  // one tile ahead
      for (int j = t0; ok && j < t1; ++j, ++kc) {
        const int st = kc % STAGES, at = next, row = (j * BKV) & (page - 1);
        const uint32_t ph = (kc / STAGES) & 1;
        if (j + 1 < t1) next = page_of(b, L, j + 1);
        const int off = st * TILE + ch * CHUNK + box * rows * 128;
        ok = wait_all(&t.k_empty[st], ph ^ 1u, 0x52u);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&t.k_full[st], TILE);
        __syncwarp();
        if (mine) tma_load_4d(sK + off, &tmK, &t.k_full[st], ch * 64, g, row, at);
        k_issued |= 1u << st;
        k_par = (k_par & ~(1u << st)) | (ph << st);
        // the unit's Q behind its first K tile: that place is free earlier
        for (int x = 0; ok && j == t0 && x < tiles_q; ++x, ++qc) {
          const int qs = qc & 1;
          const uint32_t qph = (qc >> 1) & 1;
          ok = wait_all(&t.q_empty[qs], qph ^ 1u, 0x51u);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&t.q_full[qs], p.tq * p.G * D * 2);
            for (int e = 0; e < CH; ++e)
              tma_load_3d(sQ + qs * Gm::Q_TILE + e * Gm::Q_CHUNK, &tmQ, &t.q_full[qs], e * 64, g * p.G,
                          row0 + x * p.tq);
          }
          q_issued |= 1u << qs;
          q_par = (q_par & ~(1u << qs)) | (qph << qs);
        }
        if (!ok) break;
        ok = wait_all(&t.v_empty[st], ph ^ 1u, 0x53u);
        if (!ok) break;
        const bool tail = (L & (BKV - 1)) && j == L / BKV;
        uint64_t *bar = tail ? &t.v_raw[st] : &t.v_full[st];
        if (lane == 0) mbar_arrive_expect_tx(bar, TILE);
        __syncwarp();
        if (mine) tma_load_4d(sV + off, &tmV, bar, ch * 64, g, row, at);
        v_issued |= 1u << st;
        v_raw = (v_raw & ~(1u << st)) | (static_cast<uint32_t>(tail) << st);
        v_par = (v_par & ~(1u << st)) | (ph << st);
        raw_par ^= static_cast<uint32_t>(tail) << st;  // phases of v_raw used so far
      }
    }
    if (*abort_flag && lane == 0) {
      for (int i = 0; i < 2; ++i)
        if (q_issued & (1u << i)) mbar_drain(&t.q_full[i], (q_par >> i) & 1u, p.status);
      for (int i = 0; i < STAGES; ++i) {
        if (k_issued & (1u << i)) mbar_drain(&t.k_full[i], (k_par >> i) & 1u, p.status);
        if (v_issued & (1u << i)) {  // the stage's last copy
          if (v_raw & (1u << i)) mbar_drain(&t.v_raw[i], ((raw_par >> i) & 1u) ^ 1u, p.status);
          else mbar_drain(&t.v_full[i], (v_par >> i) & 1u, p.status);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LOW));
    // ---------------- MMA: the whole warp runs the loop, one elected lane issues
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, BKV, 0, 0);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 0, 1);
    auto wait_all = [&](uint64_t *bar, uint32_t parity, uint32_t where) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, p.wait_ns, where));
    };
    int qc = 0, kc = 0, units = 0;
    uint32_t used[2] = {0, 0};  // PVs issued per x
    bool ok = true;
    // S_x of the K tile in ring place `k` with the Q tile in place `q`, the q-th and k-th loaded
    auto issue_s = [&](int x, int q, int k) -> bool {
      const int st = k % STAGES, qs = q & 1;
      if (!wait_all(&t.q_full[qs], (q >> 1) & 1, 0x54u)) return false;
      if (!wait_all(&t.k_full[st], (k / STAGES) & 1, 0x55u)) return false;
      tc_fence_after();
      const uint32_t k_addr = smem_u32(sK + st * TILE), q_addr = smem_u32(sQ + qs * Gm::Q_TILE);
#pragma unroll
      for (int kk = 0; kk < 4 * CH; ++kk) {
        const uint64_t a = sdesc_k_sw128(q_addr + (kk >> 2) * Gm::Q_CHUNK) + 2 * (kk & 3);
        const uint64_t b = sdesc_k_sw128(k_addr + (kk >> 2) * CHUNK) + 2 * (kk & 3);
        mma_bf16_ss_w(tmem + x * BKV, a, b, idesc_s, kk > 0);
      }
      tc_commit_w(&t.s_full[x]);
      return true;
    };
    // O_x (+)= P_x V in two halves of 64 slots, each as soon as the softmax has stored it
    auto issue_pv = [&](int x, int k, bool fresh) -> bool {
      const int st = k % STAGES;
      if (!wait_all(&t.v_full[st], (k / STAGES) & 1, 0x56u)) return false;
      const uint32_t v_addr = smem_u32(sV + st * TILE);
      for (int half = 0; half < 2; ++half) {
        if (!wait_all(&t.p_ready[2 * x + half], used[x] & 1, 0x57u)) return false;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int kk = 4 * half + i;
          mma_bf16_ts_w(tmem + 256 + x * 128, tmem + x * BKV + kk * 8, sdesc_mn_sw128(v_addr + kk * 16 * 128, CHUNK),
                        idesc_pv, !(fresh && kk == 0));
        }
      }
      tc_commit_w(&t.o_done[x]);
      ++used[x];
      return true;
    };
    for (int item = 0; ok; ++item) {
      const Item *it = take(item);
      if (!it) break;
      const int t0 = uniform(it->t0), n = uniform(it->t1) - t0;
      const bool two = MODE != STEP && uniform(it->two) != 0;
      // tiles of x = 0 when it has a Q tile of its own: at least one, if n is
      const int n_a = max(min(uniform(it->a_end) - t0, n), 0);
      give_back(item);
      if (n <= 0) continue;
      bool first_pv = true;
      auto o_is_free = [&]() -> bool {  // before the piece's first PV: the softmax has read the last piece's O
        const bool first = first_pv;
        first_pv = false;
        return !first || wait_all(&t.o_free, (units & 1) ^ 1, 0x58u);
      };
      if (two) {
        for (int x = 0; ok && x < 2; ++x) {
          const int nx = x ? n : n_a;
          if (nx > 0) ok = issue_s(x, qc + x, kc);
          else ok = wait_all(&t.q_full[(qc + x) & 1], ((qc + x) >> 1) & 1, 0x54u);  // loaded all the same
          if (ok && nx <= 1) tc_commit_w(&t.q_empty[(qc + x) & 1]);
        }
        if (ok) tc_commit_w(&t.k_empty[kc % STAGES]);
        for (int i = 0; ok && i < n; ++i) {
          for (int x = 0; ok && x < 2; ++x) {
            const int nx = x ? n : n_a;
            if (i >= nx) continue;
            ok = o_is_free() && issue_pv(x, kc + i, i == 0);
            if (ok && i + 1 < nx) {
              ok = issue_s(x, qc + x, kc + i + 1);
              if (ok && i + 2 == nx) tc_commit_w(&t.q_empty[(qc + x) & 1]);
            }
          }
          if (!ok) break;
          tc_commit_w(&t.v_empty[(kc + i) % STAGES]);
          if (i + 1 < n) tc_commit_w(&t.k_empty[(kc + i + 1) % STAGES]);
        }
        qc += 2;
      } else {
        for (int i = -2; ok && i < n; ++i) {
          if (i >= 0) {
            ok = o_is_free() && issue_pv(i & 1, kc + i, i < 2);
            if (ok) tc_commit_w(&t.v_empty[(kc + i) % STAGES]);
          }
          if (ok && i + 2 < n) {
            ok = issue_s(i & 1, qc, kc + i + 2);
            if (ok) tc_commit_w(&t.k_empty[(kc + i + 2) % STAGES]);
            if (ok && i + 3 == n) tc_commit_w(&t.q_empty[qc & 1]);
          }
        }
        qc += 1;
      }
      kc += n;
      ++units;
    }
    tc_commit_w(&t.drain);
    mbar_drain(&t.drain, 0, p.status);
    __syncwarp();
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LOW));
    if (warp == 2) {
      int kc = 0;
      uint32_t par = 0;  // per stage, the parity of its next such tile
      bool ok = true;
      for (int i = 0; ok; ++i) {
        const Item *it = take(i);
        if (!it) break;
        const int n = it->t1 - it->t0, L = it->L, from = L & (BKV - 1), at = L / BKV - it->t0;
        give_back(i);
        if (from && at >= 0 && at < n) {
          const int st = (kc + at) % STAGES;
          ok = __all_sync(0xffffffffu, mbar_wait_long(&t.v_raw[st], (par >> st) & 1u, abort_flag, p.status,
                                                      p.wait_ns, 0x5Au));
          if (!ok) break;
          par ^= 1u << st;
          // a row's 128 bytes stay its own under the swizzle
          for (int ch = 0; ch < CH; ++ch) {
            uint4 *rows = reinterpret_cast<uint4 *>(sV + st * TILE + ch * CHUNK + from * 128);
            for (int e = lane; e < (BKV - from) * 8; e += 32) rows[e] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&t.v_full[st]);
        }
        kc += max(n, 0);
      }
    } else if (lane == 0) {
      walk(t, p);
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_HIGH));
    // ---------------- softmax: warps 4..7 x = 0, warps 8..11 x = 1
    const int x = (warp - 4) >> 2;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const int rt = r / p.G, rh = r - rt * p.G;  // this row's token of the tile and head of the group
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t s_col = x * BKV;
    const float c2 = p.scale_log2;
    // this row's O_x by `factor`
    auto rescale_o = [&](float factor) {
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(lane_base + 256 + x * 128 + c * 32, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
        tmem_st32(lane_base + 256 + x * 128 + c * 32, o);
      }
      tmem_st_wait();
    };
    // For units of at most 16 rows: thread t has rows t / 4 and t / 4 + 8 of
    // every tile, a quarter of their columns each.
    const int na = (lane >> 2) / p.G, nb = ((lane >> 2) + 8) / p.G;  // their tokens
    uint32_t used = 0, joins = 0;  // tiles processed, exchanges with the other warpgroup
    bool ok = quad < WARPS;
    for (int item = 0; ok; ++item) {
      const Item *it = take(item);
      if (!it) break;
      // what is needed behind the key loop is read from the item again there
      int t0, t1, step, own_tiles, mask_from, lim;
      bool live, two;
      {
        const PlanSeq s{it->n, it->L};
        const int tok0 = it->tok0;
        two = MODE != STEP && it->two != 0;
        const int shift = two ? x * p.tq : 0;  // this tile's first token in the window
        live = rt < p.tq && tok0 + shift + rt < s.n;
        lim = live ? plan_visible(s, tok0 + shift + rt + 1) : 0;
        mask_from = plan_visible(s, tok0 + shift + 1);
        t0 = it->t0;
        t1 = it->t1;
        const int n = max(t1 - t0, 0);
        if (two) {
          const int n_a = max(min(it->a_end, t1) - t0, 0);
          own_tiles = x ? n : n_a;
          step = 1;
        } else {
          own_tiles = (n + 1 - x) >> 1;
          step = 2;
        }
      }
      const bool any_live = __any_sync(0xffffffffu, live);
      const bool few = MODE == STEP || (MODE == FEW && !two && (it->n - it->tok0) * p.G <= 16);
      float m_run = -INFINITY, l = 0.f;
      int j0 = (t0 + (step == 2 ? x : 0)) * BKV;
      if (few && quad == 0) {
        // At most 16 rows: with a thread per row a warp would walk 128 columns
        // with most of its lanes idle, and the key tile would wait for it (one
        // row over 128K slots: 102.4 us against 103.6, with pages of 16 slots
        // 115 against 132).
        const PlanSeq s{it->n, it->L};
        const int tok0 = it->tok0, left = min(s.n - tok0, p.tq);
        const int lim_a = na < left ? plan_visible(s, tok0 + na + 1) : 0;
        const int lim_b = nb < left ? plan_visible(s, tok0 + nb + 1) : 0;
        float m2[2] = {-INFINITY, -INFINITY}, l2[2] = {0.f, 0.f};
        const int my = 2 * (lane & 3);
        for (int i = 0; i < own_tiles; ++i, j0 += 2 * BKV) {
          const uint32_t u = used + i;
          ok = __all_sync(0xffffffffu, mbar_wait(&t.s_full[x], u & 1, abort_flag, p.status, p.wait_ns, 0x5Bu));
          if (!ok) break;
          tc_fence_after();
          uint32_t xr[64];
          tmem_ld_rows16(lane_base + s_col, xr);
          tmem_ld_wait();
          if (EXACT && p.scores) {
            // the rows' scores as they are: a slot past a row's limit is not read again
            const int64_t row =
                (static_cast<int64_t>(it->first + tok0) * p.Hq + it->g * p.G) * p.score_stride + j0 + my;
            const int64_t row_a = row + (static_cast<int64_t>(na) * p.Hq + (lane >> 2) - na * p.G) * p.score_stride;
            const int64_t row_b = row + (static_cast<int64_t>(nb) * p.Hq + (lane >> 2) + 8 - nb * p.G) * p.score_stride;
#pragma unroll
            for (int e = 0; e < 64; e += 2)
              if ((e & 2) ? nb < left : na < left)
                *reinterpret_cast<uint2 *>(p.scores + ((e & 2) ? row_b : row_a) + (e >> 2) * 8) =
                    make_uint2(xr[e], xr[e + 1]);
          }
          if (j0 + BKV > mask_from) {
#pragma unroll
            for (int e = 0; e < 64; ++e) {
              const int col = (e >> 2) * 8 + my + (e & 1);
              if (col >= ((e & 2) ? lim_b : lim_a) - j0) xr[e] = 0xff800000u;  // -inf
            }
          }
          float f2[2];
          bool need = false;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float a = __uint_as_float(xr[2 * h]), b = __uint_as_float(xr[2 * h + 1]);
#pragma unroll
            for (int e = 4; e < 64; e += 8) {
              a = max3_nan(a, __uint_as_float(xr[e + 2 * h]), __uint_as_float(xr[e + 2 * h + 1]));
              if (e + 4 < 64) b = max3_nan(b, __uint_as_float(xr[e + 4 + 2 * h]), __uint_as_float(xr[e + 5 + 2 * h]));
            }
            float top = max_nan(a, b);
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2)) * c2;
            const float m_new = max_nan(m2[h], top);
            f2[h] = 1.f;
            if ((h ? lim_b : lim_a) > 0 && !(m_new <= m2[h] + RESCALE_THRESHOLD)) {
              need = true;
              f2[h] = m2[h] == -INFINITY ? 0.f : ex2(m2[h] - m_new);
              m2[h] = m_new;
              l2[h] *= f2[h];
            }
          }
          if (__any_sync(0xffffffffu, need) && i > 0) {
            ok = __all_sync(0xffffffffu,
                            mbar_wait(&t.o_done[x], (u - 1) & 1, abort_flag, p.status, p.wait_ns, 0x5Cu));
            if (!ok) break;
            tc_fence_after();
            const float fa = __shfl_sync(0xffffffffu, f2[0], (lane & 7) * 4);
            const float fb = __shfl_sync(0xffffffffu, f2[1], (lane & 7) * 4);
            rescale_o(lane < 8 ? fa : fb);
          }
          const uint64_t cc = f2pack(c2, c2);
          uint64_t mm[2], s2[2] = {0ull, 0ull};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float neg = m2[h] == -INFINITY ? 0.f : -m2[h];
            mm[h] = f2pack(neg, neg);
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int h = e & 1, at = (half * 8 + (e >> 1)) * 4 + 2 * h;
              float a0, a1;
              f2unpack(f2fma(f2pack(__uint_as_float(xr[at]), __uint_as_float(xr[at + 1])), cc, mm[h]), a0, a1);
              a0 = ex2(a0);
              a1 = ex2(a1);
              s2[h] = f2add(s2[h], f2pack(a0, a1));
              pk[e] = pack_bf16x2(a0, a1);
            }
            tmem_st_rows16(lane_base + s_col + half * 32, pk);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive_warp(&t.p_ready[2 * x + half]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float a, b;
            f2unpack(s2[h], a, b);
            l2[h] += a + b;
          }
        }
        // back to a thread per row
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          l2[h] += __shfl_xor_sync(0xffffffffu, l2[h], 1);
          l2[h] += __shfl_xor_sync(0xffffffffu, l2[h], 2);
          const float mr = __shfl_sync(0xffffffffu, m2[h], (lane & 7) * 4);
          const float lr = __shfl_sync(0xffffffffu, l2[h], (lane & 7) * 4);
          if ((lane >> 3) == h) {
            m_run = mr;
            l = lr;
          }
        }
      } else if (MODE != STEP) {
        for (int i = 0; i < own_tiles; ++i, j0 += step * BKV) {
          const uint32_t u = used + i;
          ok = __all_sync(0xffffffffu, mbar_wait(&t.s_full[x], u & 1, abort_flag, p.status, p.wait_ns, 0x5Bu));
          if (!ok) break;
          if (!any_live) {  // a warp of padding rows: P may be anything
            tc_fence_before();
            mbar_arrive_warp(&t.p_ready[2 * x]);
            mbar_arrive_warp(&t.p_ready[2 * x + 1]);
            continue;
          }
          tc_fence_after();
          uint32_t xr[BKV];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            tmem_ld32(lane_base + s_col + c * 32, *reinterpret_cast<uint32_t(*)[32]>(xr + 32 * c));
          tmem_ld_wait();
          if (MODE == FEW && EXACT && p.scores && live) {
            const int64_t row = static_cast<int64_t>(it->first + it->tok0 + (two ? x * p.tq : 0) + rt) * p.Hq;
            uint4 *to = reinterpret_cast<uint4 *>(p.scores + (row + it->g * p.G + rh) * p.score_stride + j0);
#pragma unroll
            for (int e = 0; e < 32; ++e) to[e] = make_uint4(xr[4 * e], xr[4 * e + 1], xr[4 * e + 2], xr[4 * e + 3]);
          }
          if (j0 + BKV > mask_from) {  // slots past the tile's first query, past the last slot among them
            const int vis = lim - j0;
#pragma unroll
            for (int c = 0; c < BKV; ++c)
              if (c >= vis) xr[c] = 0xff800000u;  // -inf
          }
          float m8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) m8[e] = __uint_as_float(xr[e]);
#pragma unroll
          for (int c = 8; c < BKV; c += 2)
            m8[(c >> 1) & 7] = max3_nan(m8[(c >> 1) & 7], __uint_as_float(xr[c]), __uint_as_float(xr[c + 1]));
          const float mt = max3_nan(max3_nan(m8[0], m8[1], m8[2]), max3_nan(m8[3], m8[4], m8[5]),
                                    max_nan(m8[6], m8[7])) * c2;
          const float m_new = max_nan(m_run, mt);
          const bool need = live && !(m_new <= m_run + RESCALE_THRESHOLD);
          if (__any_sync(0xffffffffu, need)) {
            const float factor = (m_run == -INFINITY) ? 0.f : ex2(m_run - m_new);
            if (i > 0) {  // O_x holds the tiles so far: wait for the last of them
              ok = __all_sync(0xffffffffu,
                              mbar_wait(&t.o_done[x], (u - 1) & 1, abort_flag, p.status, p.wait_ns, 0x5Cu));
              if (!ok) break;
              tc_fence_after();
              rescale_o(factor);
            }
            l *= factor;
            m_run = m_new;
          }
          const float neg_m = (m_run == -INFINITY) ? 0.f : -m_run;
          const uint64_t cc = f2pack(c2, c2), mm = f2pack(neg_m, neg_m);
          uint64_t s4[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint64_t a2 =
                  f2fma(f2pack(__uint_as_float(xr[h * 64 + 2 * e]), __uint_as_float(xr[h * 64 + 2 * e + 1])), cc, mm);
              float e0, e1;
              if (!EXACT && e % POLY_EVERY == POLY_EVERY - 1) {
                exp2_poly2(a2, e0, e1);
              } else {
                float a0, a1;
                f2unpack(a2, a0, a1);
                e0 = ex2(a0);
                e1 = ex2(a1);
              }
              s4[e & 3] = f2add(s4[e & 3], f2pack(e0, e1));
              pk[e] = pack_bf16x2(e0, e1);
            }
            tmem_st32(lane_base + s_col + h * 32, pk);  // P over S: columns [32 h, 32 h + 32)
            if (h == 0) {
              tmem_st_wait();
              tc_fence_before();
              mbar_arrive_warp(&t.p_ready[2 * x]);
            }
          }
          {
            float q0, q1, q2, q3;
            f2unpack(f2add(s4[0], s4[1]), q0, q1);
            f2unpack(f2add(s4[2], s4[3]), q2, q3);
            l += (q0 + q1) + (q2 + q3);
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive_warp(&t.p_ready[2 * x + 1]);
        }
      }
      if (!ok) break;
      used += own_tiles;

      // ---------------- end of the piece: O_x, or both O of a unit with one Q tile, leave TMEM
      const bool any_tile = t1 > t0;
      if (any_tile) {
        // its own last PV; the other warpgroup's is known through the exchange
        // below.  (A parity wait may skip no phase: S of a tile is issued
        // after the PV before it on the same x, so that one has completed.)
        if (own_tiles > 0)
          ok = __all_sync(0xffffffffu,
                          mbar_wait(&t.o_done[x], (used - 1) & 1, abort_flag, p.status, p.wait_ns, 0x5Du));
        if (!ok) break;
        tc_fence_after();
      }
      float f0 = x == 0 ? 1.f : 0.f, f1 = x == 0 ? 0.f : 1.f;  // O = f0 O_0 + f1 O_1
      if (!two && any_tile) {
        t.xchg[joins & 1][x][r] = make_float2(m_run, l);
        tc_fence_before();
        mbar_arrive_warp(&t.x_full);
        ok = __all_sync(0xffffffffu,
                        mbar_wait(&t.x_full, joins & 1, abort_flag, p.status, p.wait_ns, 0x5Eu));
        if (!ok) break;
        tc_fence_after();
        const float2 a = t.xchg[joins & 1][0][r], b = t.xchg[joins & 1][1][r];
        ++joins;
        m_run = max_nan(a.x, b.x);
        const float top = m_run == -INFINITY ? 0.f : m_run;
        f0 = ex2(a.x - top);
        f1 = ex2(b.x - top);
        l = a.y * f0 + b.y * f1;
      }
      const int row = (two ? x * p.tq : 0) + rt;      // token inside the window
      const int tok = it->first + it->tok0 + row;     // packed row
      const int head = it->g * p.G + rh;
      const int64_t part = it->part;
      const bool whole = it->whole != 0;
      give_back(item);
      // columns this warpgroup writes: all of its own O, or its half of the joined one
      const int c0 = two ? 0 : x * (D / 64), c1 = two ? D / 32 : (x + 1) * (D / 64);
      const bool first_wg = two || x == 0;
      if (live && first_wg) {
        if (whole) {
          if (p.lse) p.lse[static_cast<int64_t>(tok) * p.Hq + head] = (m_run + log2f(l)) * LN2;
        } else if (any_tile) {
          p.part_ml[part * p.slot_rows + row * p.G + rh] = make_float2(m_run, l);
        }
      }
      const float inv = whole ? (lim == 0 ? 0.f : 1.f / l) : 1.f;
      f0 *= inv;
      f1 *= inv;
      const bool use0 = two ? x == 0 && own_tiles > 0 : any_tile;
      const bool use1 = two ? x == 1 && own_tiles > 0 : t1 - t0 > 1;
      if (any_live && (whole || any_tile)) {
#pragma unroll 1
        for (int c = c0; c < c1; ++c) {
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0.f;
          if (use0) {
            uint32_t o[32];
            tmem_ld32(lane_base + 256 + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[e]) * f0;
          }
          if (use1) {
            uint32_t o[32];
            tmem_ld32(lane_base + 384 + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = fmaf(__uint_as_float(o[e]), f1, v[e]);
          }
          if (!live) continue;
          if (whole) {
            if (lim == 0) {  // no slot is visible
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = 0.f;
            }
            uint4 *dst = reinterpret_cast<uint4 *>(p.o + tok * p.o_stride + head * D + c * 32);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              dst[q] = make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                                  pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
          } else {
            float *dst = p.part_o + (part * p.slot_rows + row * p.G + rh) * D + c * 32;
#pragma unroll
            for (int q = 0; q < 4; ++q) store_8(dst + 8 * q, v + 8 * q);
          }
        }
      }
      if (any_tile) {
        tc_fence_before();
        mbar_arrive_warp(&t.o_free);
      }
    }
  }
  // what this CTA's ranges leave for the combine kernel
  if (threadIdx.x < p.max_groups && !p.whole) {
    const int group = threadIdx.x, heads = group < t.groups ? heads_of(t, p, group) : 0, rg = blockIdx.x;
    PlanCut cut{};
    cut.total = heads > 0 ? t.before[p.c.B] * heads : 0;
    const int nr = plan_ranges(cut.total, gridDim.x);
    if (rg < nr && cut.total > 0) {
      PlanCursor cur;
      plan_open(cur, t.seq, t.before, p.c.B, shape_of(p), heads, plan_cut(cut.total, nr, rg), 1);
      const PlanSeq s = t.seq[cur.b];
      cut = PlanCut{cut.total, nr,    cur.b, cur.p, group * t.group_heads + cur.g, cur.off, cur.c, s.n, s.L,
                    t.first[cur.b]};
    }
    p.cuts[group * gridDim.x + rg] = cut;
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Joins the pieces of the unit whose first cut is in front of range
// blockIdx.x + 1 of group blockIdx.y: O = sum_i 2^(m_i - m) O_i / sum_i
// 2^(m_i - m) l_i, the pieces in order.  A chain of dependent loads (the cut,
// the statistics, the rows), so a warp takes JOIN_ROWS rows at once.  Launched
// while the attention still runs (its CTAs take the places of those that
// ended), and waits for it.
constexpr int JOIN_WARPS = 8;

template <int D, int ROWS, int DEEP>
__global__ void __launch_bounds__(32 * JOIN_WARPS) paged_combine_kernel(const __grid_constant__ Params p, int ctas) {
  const int range = blockIdx.x + 1, group = blockIdx.y;
  constexpr int E = D / 32;
  using Vec = std::conditional_t<D == 128, float4, float2>;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PlanCut cut = p.cuts[group * ctas + range];
  if (!plan_first_cut(cut, range)) return;
  const PlanSeq s{cut.n, cut.L};
  const int w = p.w, tok0 = cut.p * w, g = cut.g;
  const int rows = min(w, s.n - tok0) * p.G;
  const int tiles = (plan_visible(s, tok0 + w) + BKV - 1) / BKV;
  const int lane = threadIdx.x & 31;
  // where piece i of this unit lies, or -1 if it has no tile; `last`: whether it ends the unit
  auto piece = [&](int i, bool &last) -> int64_t {
    int rg, slot, off, end, t0, t1;
    plan_piece_of(cut, range, i, rg, slot, off, end);
    last = end == cut.c;
    if (off == cut.c) return -1;
    plan_tiles(off, end, cut.c, tiles, t0, t1);
    return t0 < t1 ? ((static_cast<int64_t>(group) * ctas + rg) * 2 + slot) * p.slot_rows : -1;
  };
  const int warps = static_cast<int>(gridDim.z) * JOIN_WARPS;
  for (int row0 = blockIdx.z * JOIN_WARPS + (threadIdx.x >> 5); row0 < rows; row0 += warps * ROWS) {
    float m[ROWS], l[ROWS], acc[ROWS][E];
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
      m[q] = -INFINITY;
      l[q] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[q][e] = 0.f;
    }
    bool done = false;
    for (int i0 = 0; !done; i0 += 32) {  // 32 pieces at a time: lane i has the statistics of piece i0 + i
      bool last;
      const int64_t at = piece(i0 + lane, last);
      done = __any_sync(0xffffffffu, last);
      const int pieces = 32 - __clz(__ballot_sync(0xffffffffu, at >= 0));
      float2 ml[ROWS];
#pragma unroll
      for (int q = 0; q < ROWS; ++q) {
        const int row = row0 + q * warps;
        ml[q] = at >= 0 && row < rows ? p.part_ml[at + row] : make_float2(-INFINITY, 0.f);
      }
      float f[ROWS];
      uint32_t live[ROWS];  // pieces of which the row sees nothing are skipped: their O may be anything
#pragma unroll
      for (int q = 0; q < ROWS; ++q) {
        float top = ml[q].x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float mn = max_nan(m[q], top), zero = mn == -INFINITY ? 0.f : mn, keep = ex2(m[q] - zero);
        f[q] = ex2(ml[q].x - zero);
        float part = ml[q].y * f[q];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        l[q] = l[q] * keep + part;
        m[q] = mn;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[q][e] *= keep;
        live[q] = __ballot_sync(0xffffffffu, ml[q].x != -INFINITY);
      }
      for (int j = 0; j < pieces; j += DEEP) {
        Vec v[DEEP][ROWS];
#pragma unroll
        for (int i = 0; i < DEEP; ++i) {
          const int64_t from = __shfl_sync(0xffffffffu, at, (j + i) & 31);
#pragma unroll
          for (int q = 0; q < ROWS; ++q) {
            v[i][q] = Vec{};
            if (j + i < pieces && ((live[q] >> ((j + i) & 31)) & 1u))
              v[i][q] = *reinterpret_cast<const Vec *>(p.part_o + (from + row0 + q * warps) * D + lane * E);
          }
        }
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
#pragma unroll
          for (int q = 0; q < ROWS; ++q) {
            const float fi = __shfl_sync(0xffffffffu, f[q], (j + i) & 31);
            if (j + i < pieces && ((live[q] >> ((j + i) & 31)) & 1u)) {
#pragma unroll
              for (int e = 0; e < E; ++e)
                acc[q][e] = fmaf(reinterpret_cast<const float *>(&v[i][q])[e], fi, acc[q][e]);
            }
          }
      }
    }
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
      const int row = row0 + q * warps;
      if (row >= rows) break;
      const int tok = cut.first + tok0 + row / p.G, head = g * p.G + row % p.G;
      const bool none = plan_visible(s, tok0 + row / p.G + 1) == 0;
      const float inv = none ? 0.f : 1.f / l[q];
      __nv_bfloat16 *o = p.o + tok * p.o_stride + head * D + lane * E;
      uint32_t packed[E / 2];
#pragma unroll
      for (int e = 0; e < E; e += 2) packed[e / 2] = pack_bf16x2(acc[q][e] * inv, acc[q][e + 1] * inv);
      if (E == 4) *reinterpret_cast<uint2 *>(o) = make_uint2(packed[0], packed[E / 2 - 1]);
      else *reinterpret_cast<uint32_t *>(o) = packed[0];
      if (lane == 0 && p.lse)
        p.lse[static_cast<int64_t>(tok) * p.Hq + head] = none ? -INFINITY : (m[q] + log2f(l[q])) * LN2;
    }
  }
}

struct Scratch {
  float *part_o;
  float2 *part_ml;
  PlanCut *cuts;
  size_t bytes;
};

Scratch carve(void *base, int d, int groups, int ctas, int slot_rows) {
  char *at = static_cast<char *>(base);
  const size_t slots = static_cast<size_t>(groups) * ctas * 2 * slot_rows;
  Scratch s;
  s.part_o = reinterpret_cast<float *>(at);
  size_t off = Carver::round(slots * d * sizeof(float));
  s.part_ml = reinterpret_cast<float2 *>(at + off);
  off += Carver::round(slots * sizeof(float2));
  s.cuts = reinterpret_cast<PlanCut *>(at + off);
  off += Carver::round(sizeof(PlanCut) * groups * ctas);
  s.bytes = off;
  return s;
}


template <int D, bool EXACT, Mode MODE>
spts_status launch(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const Params &p, int ctas,
                   cudaStream_t s) {
  SPTS_TRY((allow_smem<paged_attn_kernel<D, EXACT, MODE>>(smem_bytes<D, MODE>())));
  paged_attn_kernel<D, EXACT, MODE><<<ctas, THREADS, smem_bytes<D, MODE>(), s>>>(tq, tk, tv, p);
  note_launch();
  SPTS_CUDA_TRY(cudaGetLastError());
  if (ctas > 1 && !p.whole) {
    // Few units are cut into many pieces each: a row to a warp and eight pieces
    // on their way, as for steps (28 rows of 2 heads over 4574 slots, 74
    // pieces per unit: 26 us, and 47 with four rows to a warp and two pieces);
    // CTAs per unit: one turn of its warps for the largest window.
    const int64_t units = (static_cast<int64_t>(p.T) / p.w + p.c.B) * p.c.Hkv;
    const bool deep = MODE != FULL || units * 8 <= ctas;
    const int most = (p.T < p.w ? p.T : p.w) * p.G, turn = JOIN_WARPS * (deep ? 1 : 4);
    const int split = MODE == FULL ? (most + turn - 1) / turn : 1;
    SPTS_TRY(launch_behind(deep ? paged_combine_kernel<D, 1, 8> : paged_combine_kernel<D, 4, 2>,
                           dim3(ctas - 1, p.max_groups, split), 32 * JOIN_WARPS, s, 0, p, ctas));
  }
  return SPTS_OK;
}

}  // namespace

spts_status paged_q_map(const PagedView &c, const PagedAttnArgs &a, int tokens, CUtensorMap *q) {
  const uint64_t D = c.d, G = a.Hq / c.Hkv;
  const uint64_t dims[3] = {D, static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(a.T)};
  const uint64_t strides[2] = {D * 2, static_cast<uint64_t>(a.q_stride) * 2};
  const uint32_t box[3] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(tokens)};
  return make_tmap(q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

spts_status paged_kv_map(const PagedView &c, const void *pages, CUtensorMap *map) {
  const uint64_t D = c.d, page = uint64_t(1) << c.page_shift;
  const uint64_t dims[4] = {D, static_cast<uint64_t>(c.Hkv), page, static_cast<uint64_t>(c.num_pages)};
  const uint64_t strides[3] = {D * 2, static_cast<uint64_t>(c.Hkv) * D * 2, static_cast<uint64_t>(c.page_stride) * 2};
  const uint32_t box[4] = {64, 1, static_cast<uint32_t>(page < PLAN_TILE ? page : PLAN_TILE), 1};
  return make_tmap(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pages, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

namespace {

// How a call is launched, from the sizes that the host knows.
struct Shape {
  Mode mode;
  int whole;      // units are dealt out whole: no scratch, no combine kernel
  int tq, w;      // tokens of a Q tile and of a window
  int groups;     // head groups that the sizes can call for (up to MAX_GROUPS: 40 MB of scratch each)
  int slot_rows;  // rows of a partial result
};
constexpr int MAX_GROUPS = 4;
constexpr int64_t WHOLE_SLOTS = 1024;

// 16 rows of a KV head or less per sequence on average.
bool few_rows(int B, int64_t T, int G) { return T * G <= 16 * static_cast<int64_t>(B); }

Shape shape_of(int B, int64_t T, int64_t slots, int Hq, int Hkv, int d, int ctas) {
  const int G = Hq / Hkv;
  // With tables of up to WHOLE_SLOTS slots units are not cut: windows of prompts
  // would leave many pieces to join (whole against cut, us per call in a row: 61
  // prompts of up to 235 tokens 46, 81; one of 1000 24, 40; 8 of 400 to 1000 80,
  // 107).  Steps would be a tenth faster cut (one row over 517 slots 14.0, 12.8;
  // 300 rows over up to 1001 135, 121).
  const int whole = slots <= WHOLE_SLOTS;
  // One token per sequence or less on average: steps of decoding.  (Sequences
  // with many tokens come out right, in windows of few.)
  if (T <= B && G <= 16) return Shape{STEP, whole, 16 / G, 16 / G, whole ? 0 : 1, 16};
  const int tq = 128 / G, w = 2 * tq;
  const int64_t windows = T / w + B;
  const int groups = plan_groups(static_cast<int64_t>(B) * slots * Hkv * d * 4, windows * (slots + PLAN_TWO) * Hkv,
                                 ctas, Hkv, MAX_GROUPS);
  return Shape{few_rows(B, T, G) ? FEW : FULL, whole, tq, w, whole ? 0 : groups, 256};
}

int64_t score_stride(int64_t slots) { return (slots + BKV - 1) / BKV * BKV; }

}  // namespace

// With few rows the attention leaves its scores (G fp32 values per slot and
// KV head, against d bf16 values of K for computing them again), as long as
// they stay below SCORE_BYTES.
constexpr size_t SCORE_BYTES = size_t(256) << 20;
size_t paged_scores_bytes(int B, int64_t T, int64_t slots, int Hq, int Hkv) {
  const size_t bytes = static_cast<size_t>(T) * Hq * score_stride(slots) * sizeof(float);
  return few_rows(B, T, Hq / Hkv) && bytes <= SCORE_BYTES ? bytes : 0;
}

size_t paged_attn_scratch_bytes(int B, int64_t T, int64_t slots, int Hq, int Hkv, int d) {
  const int ctas = num_sms();
  const Shape sh = shape_of(B, T, slots, Hq, Hkv, d, ctas);
  return carve(nullptr, d, sh.groups, ctas, sh.slot_rows).bytes;
}

spts_status launch_paged_attention(const PagedView &c, const PagedAttnArgs &a, cudaStream_t s) {
  if (a.T == 0) return SPTS_OK;
  const int D = c.d, ctas = num_sms();
  const int64_t slots = static_cast<int64_t>(c.max_pages) << c.page_shift;
  const Shape sh = shape_of(c.B, a.T, slots, a.Hq, c.Hkv, D, ctas);
  CUtensorMap q_map, k_map, v_map;
  SPTS_TRY(paged_q_map(c, a, sh.tq, &q_map));
  SPTS_TRY(paged_kv_map(c, c.k, &k_map));
  SPTS_TRY(paged_kv_map(c, c.v, &v_map));
  const Scratch sc = carve(a.scratch, D, sh.groups, ctas, sh.slot_rows);
  Params p{};
  p.c = c;
  p.cu = a.cu;
  p.T = static_cast<int>(a.T);
  p.Hq = a.Hq;
  p.G = a.Hq / c.Hkv;
  p.tq = sh.tq;
  p.w = sh.w;
  p.slot_rows = sh.slot_rows;
  p.whole = sh.whole;
  p.max_groups = sh.groups;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.o = static_cast<__nv_bfloat16 *>(a.o);
  p.o_stride = a.o_stride;
  p.lse = a.lse;
  p.part_o = sc.part_o;
  p.part_ml = sc.part_ml;
  p.cuts = sc.cuts;
  p.status = a.status;
  p.wait_ns = wait_limit_ns();
  p.scores = a.weights && a.scores ? a.scores : nullptr;
  p.score_stride = score_stride(slots);
  using Launch = spts_status (*)(const CUtensorMap &, const CUtensorMap &, const CUtensorMap &, const Params &, int,
                                 cudaStream_t);
  static constexpr Launch launches[2][2][3] = {
      {{launch<64, false, FULL>, launch<64, false, FEW>, launch<64, false, STEP>},
       {launch<64, true, FULL>, launch<64, true, FEW>, launch<64, true, STEP>}},
      {{launch<128, false, FULL>, launch<128, false, FEW>, launch<128, false, STEP>},
       {launch<128, true, FULL>, launch<128, true, FEW>, launch<128, true, STEP>}}};
  SPTS_TRY(launches[D == 128][a.lse != nullptr][sh.mode](q_map, k_map, v_map, p, ctas, s));
  if (a.weights == nullptr) return SPTS_OK;
  return p.scores ? launch_stored_weights(c, a, p.score_stride, s) : launch_paged_weights(c, a, k_map, s);
}

}  // namespace spts
