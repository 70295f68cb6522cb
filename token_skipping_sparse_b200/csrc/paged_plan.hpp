// paged_plan.hpp -- how the attention over the paged cache is shared out
// among the CTAs: plain integer arithmetic, the same on the device and on
// the host.
//
// Work is counted in key slots.  A unit is a window of w new tokens of one
// sequence (two Q tiles of w / 2 tokens) and one KV head; window p of a
// sequence with n new tokens behind `base` earlier ones costs
// base + (p + 1) w slots, which is what its last token sees (a little more in
// the last window), so the cost of the first p windows has a closed form and
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

SPTS_HD int plan_min(int a, int b) { return a < b ? a : b; }
SPTS_HD int plan_max(int a, int b) { return a > b ? a : b; }

struct PlanSeq {
  int n, L;  // new tokens, cached tokens (the new ones included)
};

SPTS_HD int plan_windows(int n, int w) { return (n + w - 1) / w; }
SPTS_HD int plan_base(const PlanSeq &s) { return plan_max(s.L - s.n, 0); }
// Cost of the first p windows of a sequence, for one head.
SPTS_HD int64_t plan_cost(int base, int p, int w) {
  return static_cast<int64_t>(p) * base + static_cast<int64_t>(w) * p * (p + 1) / 2;
}

// Range r of `nr` equal ranges of `total`.
SPTS_HD int64_t plan_cut(int64_t total, int nr, int r) {
  const int64_t q = total / nr, m = total % nr;
  return q * r + (r < m ? r : m);
}

// Where a position falls: window p and head g of a sequence, `off` slots into
// that unit's cost c.
struct PlanUnit {
  int p, g;
  int off, c;
};

// y: position inside the sequence's units of one head group of `heads` heads.
SPTS_HD PlanUnit plan_locate(const PlanSeq &s, int w, int heads, int64_t y) {
  const int base = plan_base(s);
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
  u.g = static_cast<int>(z / u.c);
  u.off = static_cast<int>(z - static_cast<int64_t>(u.g) * u.c);
  return u;
}

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

// Ranges a group of total cost `total` is cut into: none shorter than a tile.
SPTS_HD int plan_ranges(int64_t total, int ctas) {
  const int64_t r = total / PLAN_TILE;
  return r < 1 ? 1 : (r < ctas ? static_cast<int>(r) : ctas);
}

}  // namespace spts
