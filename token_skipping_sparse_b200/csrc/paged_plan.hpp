// paged_plan.hpp -- how the attention over the paged cache is shared out
// among the CTAs: plain integer arithmetic, the same on the device and on
// the host.
//
// Work is counted in key slots.  A unit is a window of w new tokens of one
// sequence (one or two Q tiles) and one KV head; window p of a
// sequence with n new tokens behind others costs base + (p + 1) w slots: what
// its last token sees (a little more in the last window) and a constant for
// what a unit costs beyond its tiles, so the cost of the first p windows has a closed form and
// no list of units is needed.  Units are ordered by (head group, sequence,
// window, head); a group's units, end to end, are cut into equal ranges, one
// per CTA, wherever the cuts fall.  A unit that a cut divides is put together
// again from its pieces by the combine kernel.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SPTS_HD __host__ __device__ __forceinline__
#else
#define SPTS_HD inline
#endif

namespace spts {

constexpr int PLAN_TILE = 128;  // key slots of one tile
// What a unit costs beyond its tiles (its Q, the end of its pipeline, its
// output), in key slots: PLAN_ONE with one Q tile, PLAN_TWO with two.
#ifndef SPTS_PLAN_ONE
#define SPTS_PLAN_ONE 128
#endif
#ifndef SPTS_PLAN_TWO
#define SPTS_PLAN_TWO 512
#endif
constexpr int PLAN_ONE = SPTS_PLAN_ONE, PLAN_TWO = SPTS_PLAN_TWO;

SPTS_HD int plan_min(int a, int b) { return a < b ? a : b; }
SPTS_HD int plan_max(int a, int b) { return a > b ? a : b; }

// Whether a row of a page table has a slot t.
SPTS_HD bool paged_has_slot(int t, int max_pages, int page_shift) {
  return t >= 0 && (t >> page_shift) < max_pages;
}

struct PlanShape {
  int w, tile;  // tokens of a window (one or two Q tiles) and of a Q tile
};

struct PlanSeq {
  int n, L;  // new tokens, cached tokens (the new ones included)
};

SPTS_HD int plan_windows(int n, int w) { return (n + w - 1) / w; }
// What every window of a sequence costs besides its own tokens.
SPTS_HD int plan_base(const PlanSeq &s, PlanShape sh) {
  return plan_max(s.L - s.n, 0) + (sh.w > sh.tile && s.n > sh.tile ? PLAN_TWO : PLAN_ONE);
}
// Cost of the first p windows of a sequence, for one head.
SPTS_HD int64_t plan_cost(int base, int p, int w) {
  return static_cast<int64_t>(p) * base + static_cast<int64_t>(w) * p * (p + 1) / 2;
}

// a / b for a >= 0, b > 0, in 32 bits where they fit (a 64-bit division takes
// the GPU several times as long).
SPTS_HD int64_t plan_div(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// Range r of `nr` equal ranges of `total`.
SPTS_HD int64_t plan_cut(int64_t total, int nr, int r) {
  const int64_t q = plan_div(total, nr), m = total - q * nr;
  return q * r + (r < m ? r : m);
}

// Where a position falls: window p and head g of a sequence, `off` slots into
// that unit's cost c.
struct PlanUnit {
  int p, g;
  int off, c;
};

// First slot that no token of [window start, window start + tokens) sees, for
// tokens counted inside the sequence's new ones.
SPTS_HD int plan_visible(const PlanSeq &s, int last_token_end) {
  return plan_max(s.L - s.n + plan_min(last_token_end, s.n), 0);
}

// Key tiles of the piece [off, end) of a unit with cost c and `tiles` tiles:
// every tile belongs to exactly one piece.
SPTS_HD void plan_tiles(int off, int end, int c, int tiles, int &t0, int &t1) {
  t0 = plan_min(tiles, (off + PLAN_TILE - 1) / PLAN_TILE);
  t1 = end == c ? tiles : plan_min(tiles, (end + PLAN_TILE - 1) / PLAN_TILE);
}

// With two Q tiles: end of the key tiles that the first one goes over in the
// piece [t0, t1) of window p.  Those it sees, and at least one of every piece that
// has any: a warpgroup without a tile would have nothing to wait for, and run
// ahead of the other one through the barrier that frees O.  (A tile that it does
// not see is masked as a whole, and its rows stay as they are.)
SPTS_HD int plan_first_end(const PlanSeq &s, PlanShape sh, int p, int t0, int t1) {
  const int sees = (plan_visible(s, p * sh.w + sh.tile) + PLAN_TILE - 1) / PLAN_TILE;
  return plan_min(t1, plan_max(sees, t0 + 1));
}

// Ranges a group of total cost `total` is cut into: none shorter than a tile.
SPTS_HD int plan_ranges(int64_t total, int ctas) {
  const int64_t r = total / PLAN_TILE;
  return r < 1 ? 1 : (r < ctas ? static_cast<int>(r) : ctas);
}


// y: position inside the sequence's units of one head group of `heads` heads.
SPTS_HD PlanUnit plan_locate(const PlanSeq &s, PlanShape sh, int heads, int64_t y) {
  const int w = sh.w, base = plan_base(s, sh);
  int lo = 0, hi = plan_windows(s.n, w) - 1;  // the window, by its first position
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (plan_cost(base, mid, w) * heads <= y) lo = mid;
    else hi = mid - 1;
  }
  PlanUnit u;
  u.p = lo;
  u.c = base + (lo + 1) * w;
  const int64_t z = y - plan_cost(base, lo, w) * heads;
  u.g = static_cast<int>(plan_div(z, u.c));
  u.off = static_cast<int>(z - static_cast<int64_t>(u.g) * u.c);
  return u;
}

// A walk over the pieces of one range.
struct PlanCursor {
  int b, p, g;   // the unit the walk stands in
  int off, c;    // how far into it, and its cost
  int64_t left;  // what is left of the range
};

struct PlanPiece {
  int b, p, g;
  int off, c;         // where in its unit it begins (at the start of a walk this may be > 0), the unit's cost
  int t0, t1, tiles;  // its key tiles, and how many the unit has
  int whole;          // the piece is the unit
  int slot;           // otherwise: where its partial result goes (0: it begins inside the unit, 1: at its start)
};

// Stands a walk at position x of a group of `heads` heads; before[b] is the
// cost of the sequences before b for one head (before[B]: of all).
SPTS_HD void plan_open(PlanCursor &cur, const PlanSeq *seq, const int64_t *before, int B, PlanShape sh, int heads,
                       int64_t x, int64_t length) {
  int lo = 0, hi = B - 1;  // the last sequence that begins at or before x and has any cost
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (before[mid] * heads <= x) lo = mid;
    else hi = mid - 1;
  }
  cur.left = length;
  cur.b = lo;
  if (length <= 0) return;
  const PlanUnit u = plan_locate(seq[lo], sh, heads, x - before[lo] * heads);
  cur.p = u.p;
  cur.g = u.g;
  cur.off = u.off;
  cur.c = u.c;
}

// The next piece, or 0 at the end of the range.
SPTS_HD int plan_next(PlanCursor &cur, const PlanSeq *seq, int B, PlanShape sh, int heads, PlanPiece &pc) {
  if (cur.left <= 0 || cur.b >= B) return 0;
  const int w = sh.w;
  const PlanSeq s = seq[cur.b];
  const int take = static_cast<int>(cur.left < cur.c - cur.off ? cur.left : cur.c - cur.off);
  pc.b = cur.b;
  pc.p = cur.p;
  pc.g = cur.g;
  pc.off = cur.off;
  pc.c = cur.c;
  pc.tiles = (plan_visible(s, (cur.p + 1) * w) + PLAN_TILE - 1) / PLAN_TILE;
  plan_tiles(cur.off, cur.off + take, cur.c, pc.tiles, pc.t0, pc.t1);
  pc.whole = take == cur.c;
  pc.slot = cur.off > 0 ? 0 : 1;
  cur.left -= take;
  if (cur.off + take == cur.c) {
    cur.off = 0;
    if (++cur.g == heads) {
      cur.g = 0;
      if (++cur.p == plan_windows(s.n, w)) {
        cur.p = 0;
        do ++cur.b;
        while (cur.b < B && seq[cur.b].n <= 0);
      }
    }
    if (cur.b < B) cur.c = plan_base(seq[cur.b], sh) + (cur.p + 1) * w;
  } else {
    cur.off += take;
  }
  return 1;
}

// Head groups (a power of two, at most `most`).  With one group the CTAs stand
// at places spread over all keys of all heads, so K and V that several units
// share must stay in L2 as a whole (2048 rows over 32K slots, 134 MB: 1.73 GB
// read from HBM with one group, 0.17 GB with four).  More groups mean more
// cuts, worth PLAN_GROUP_TILES of each CTA's tiles or more.
constexpr int64_t PLAN_GROUP_BYTES = int64_t(72) << 20;
constexpr int PLAN_GROUP_TILES = 64;
SPTS_HD int plan_groups(int64_t shared_bytes, int64_t total, int ctas, int heads, int most) {
  int groups = 1;
  while (2 * groups <= most && 2 * groups <= heads && shared_bytes > groups * PLAN_GROUP_BYTES &&
         total / PLAN_TILE >= static_cast<int64_t>(2) * groups * ctas * PLAN_GROUP_TILES)
    groups *= 2;
  return groups;
}

// What the range r leaves for the combine kernel about its first position.
struct PlanCut {
  int64_t total;  // cost of the group
  int nr;         // its ranges (0: this range is not one of them)
  int b, p, g;    // the unit at the cut (g: counted over all heads)
  int off, c;     // how far inside it the cut is (0: between two units), and the unit's cost
  int n, L, first;  // its sequence: new tokens, cached tokens, first packed row
};

// Whether the cut in front of range r is the first one inside its unit.
SPTS_HD int plan_first_cut(const PlanCut &cut, int r) {
  return r > 0 && r < cut.nr && cut.off > 0 &&
         plan_cut(cut.total, cut.nr, r) - cut.off >= plan_cut(cut.total, cut.nr, r - 1);
}

// Piece i of the unit whose first cut is in front of range r: the range that
// computed it, its slot there, and its [off, end) in the unit (empty, at the
// unit's end, past its last piece).
SPTS_HD void plan_piece_of(const PlanCut &cut, int r, int i, int &range, int &slot, int &off, int &end) {
  const int64_t start = plan_cut(cut.total, cut.nr, r) - cut.off, c = cut.c;
  range = r - 1 + i;
  slot = i == 0 ? 1 : 0;
  const int64_t o = i == 0 ? 0 : plan_cut(cut.total, cut.nr, range) - start;
  const int64_t e = plan_cut(cut.total, cut.nr, range + 1) - start;
  off = static_cast<int>(o < c ? o : c);
  end = static_cast<int>(e < c ? e : c);
}

// The accumulated weights' pass: K tiles of a head, each with the Q tiles (of tq
// tokens) that see any of its slots.  Cost of a head's first j tiles, in
// tokens, with PLAN_KEYS Q tiles for what a K tile costs by itself; the tokens
// in front of a tile's first slot do not see it.
constexpr int PLAN_KEYS = 2;
SPTS_HD int64_t plan_keys_cost(const PlanSeq &s, int tq, int64_t j) {
  const int64_t base = s.L - s.n, first = base < 0 ? 0 : base / PLAN_TILE + 1;  // the first tile some tokens miss
  int64_t cost = j * (static_cast<int64_t>(plan_windows(s.n, tq)) + PLAN_KEYS) * tq;
  if (j > first) cost -= (PLAN_TILE / 2) * (first + j - 1) * (j - first) - base * (j - first);
  return cost;
}

// The first of a head's `tiles` tiles that begins at cost x or later (`tiles`: none).
SPTS_HD int plan_keys_at(const PlanSeq &s, int tq, int tiles, int64_t x) {
  int lo = 0, hi = tiles;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (plan_keys_cost(s, tq, mid) >= x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Units whose K tiles leave warpgroups over (of four) share out their Q tiles:
// warpgroup x takes K tile x % tiles and every plan_sharers-th Q tile.
SPTS_HD int plan_sharers(int tiles, int q_tiles) { return plan_min(tiles > 2 ? 1 : 4 / tiles, q_tiles); }

}  // namespace spts
