"""The plan of the attention over the paged cache: every key tile of every unit is computed once, whatever the lengths
and the number of CTAs (CPU: the plan is plain arithmetic, compiled here for the host)."""

import ctypes as C
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "token_skipping_sparse_b200", "csrc")

SHIM = r"""
#include "paged_plan.hpp"
#include <vector>
using namespace spts;
// Walks every range of one head group as the kernel does.  rows: 9 ints per piece
// (range, b, p, g, t0, t1, tiles, whole, slot); cuts: the record of each range.
extern "C" int walk(int B, const int *n, const int *L, int w, int tile, int heads, int ctas, int *rows, int cap,
                    PlanCut *cuts) {
  const PlanShape sh{w, tile};
  std::vector<PlanSeq> seq(B);
  std::vector<int64_t> before(B + 1, 0);
  for (int b = 0; b < B; ++b) {
    seq[b] = PlanSeq{n[b], L[b]};
    before[b + 1] = before[b] + plan_cost(plan_base(seq[b], sh), plan_windows(n[b], w), w);
  }
  const int64_t total = before[B] * heads;
  const int nr = plan_ranges(total, ctas);
  int count = 0;
  for (int r = 0; r < nr; ++r) {
    const int64_t x = plan_cut(total, nr, r);
    PlanCursor cur;
    plan_open(cur, seq.data(), before.data(), B, sh, heads, x, plan_cut(total, nr, r + 1) - x);
    cuts[r] = PlanCut{total, nr, cur.b, cur.p, cur.g, cur.off, cur.c, n[cur.b], L[cur.b], 0};
    PlanPiece pc;
    while (plan_next(cur, seq.data(), B, sh, heads, pc)) {
      if (count == cap) return -1;
      const int v[9] = {r, pc.b, pc.p, pc.g, pc.t0, pc.t1, pc.tiles, pc.whole, pc.slot};
      for (int i = 0; i < 9; ++i) rows[9 * count + i] = v[i];
      ++count;
    }
  }
  return count;
}
extern "C" int first_cut(const PlanCut *cut, int r) { return plan_first_cut(*cut, r); }
extern "C" void piece_of(const PlanCut *cut, int r, int i, int *out) {
  plan_piece_of(*cut, r, i, out[0], out[1], out[2], out[3]);
}
extern "C" int64_t keys_cost(int n, int L, int tq, int64_t j) { return plan_keys_cost(PlanSeq{n, L}, tq, j); }
extern "C" int keys_at(int n, int L, int tq, int tiles, int64_t x) { return plan_keys_at(PlanSeq{n, L}, tq, tiles, x); }
extern "C" int sharers(int tiles, int q_tiles) { return plan_sharers(tiles, q_tiles); }
extern "C" void tiles_of(int off, int end, int c, int tiles, int *out) { plan_tiles(off, end, c, tiles, out[0], out[1]); }
"""


class Cut(C.Structure):
    _fields_ = [("total", C.c_int64)] + [(n, C.c_int) for n in ("nr", "b", "p", "g", "off", "c", "n", "L", "first")]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    at = tmp_path_factory.mktemp("plan")
    (at / "shim.cpp").write_text(SHIM)
    so = str(at / "plan.so")
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(at / "shim.cpp"), "-o", so], check=True)
    return C.CDLL(so)


def run(plan, n, L, w, heads, ctas, tile=None):
    B, cap = len(n), 200000
    rows = np.zeros((cap, 9), np.int32)
    cuts = (Cut * ctas)()
    arr = lambda v: (C.c_int * len(v))(*v)  # noqa: E731
    count = plan.walk(B, arr(n), arr(L), w, tile or -(-w // 2), heads, ctas, rows.ctypes.data_as(C.c_void_p), cap, cuts)
    assert count >= 0
    return rows[:count], cuts


def check(plan, n, L, w, heads, ctas, tile=None):
    rows, cuts = run(plan, n, L, w, heads, ctas, tile)
    want = {}
    for b, (m, length) in enumerate(zip(n, L)):
        for p in range(-(-m // w)):
            seen = max(length - m + min((p + 1) * w, m), 0)
            for g in range(heads):
                want[b, p, g] = -(-seen // 128)
    got, slots, whole = {}, set(), set()
    for r, b, p, g, t0, t1, tiles, w_, slot in rows.tolist():
        u = (b, p, g)
        assert tiles == want[u] and 0 <= t0 <= t1 <= tiles
        assert u not in whole
        if w_:
            assert u not in got and (t0, t1) == (0, tiles)
            whole.add(u)
        else:
            assert (r, slot) not in slots
            slots.add((r, slot))
        got.setdefault(u, []).append((t0, t1, r, slot))
    assert set(got) == set(want)
    for u, pieces in got.items():
        at = 0
        for t0, t1, _, _ in pieces:
            assert t0 == at or t0 == t1
            at = max(at, t1)
        assert at == want[u]
    # the combine kernel finds every divided unit once, and the same pieces
    found, out = {}, (C.c_int * 4)()
    nr = cuts[0].nr if n and any(n) else 0
    for r in range(nr):
        if not plan.first_cut(C.byref(cuts[r]), r):
            continue
        u = (cuts[r].b, cuts[r].p, cuts[r].g)
        assert u not in found
        pieces, i = [], 0
        while True:
            plan.piece_of(C.byref(cuts[r]), r, i, out)
            rng, slot, off, end = list(out)
            plan.tiles_of(off, end, cuts[r].c, want[u], out)
            pieces.append((out[0], out[1], rng, slot))
            i += 1
            if end == cuts[r].c:
                break
        found[u] = pieces
    assert found == {u: p for u, p in got.items() if u not in whole}


def test_one_step_of_decoding(plan):
    for L in (1, 2, 127, 128, 129, 517, 131072):
        for ctas in (1, 3, 148):
            check(plan, [1], [L], 64, 8, ctas)


def test_whole_prompts_and_chunks(plan):
    for G in (1, 2, 3, 4, 5, 7, 8, 16, 64, 128):
        w = 2 * (128 // G)
        for n, L in ((1, 1), (w, w), (w + 1, 700), (500, 500), (777, 5000), (300, 40)):
            check(plan, [n], [L], w, 2, 148)


def test_ragged_batches(plan):
    rng = np.random.default_rng(5)
    for _ in range(150):
        B = int(rng.integers(1, 40))
        n = [int(x) for x in rng.integers(0, rng.choice([2, 9, 300]), B)]
        L = [int(max(0, m + rng.integers(-3 if m else 0, rng.choice([1, 50, 4000])))) for m in n]
        w = 2 * (128 // int(rng.choice([1, 2, 3, 4, 7, 8, 32])))
        check(plan, n, L, w, int(rng.integers(1, 9)), int(rng.choice([1, 2, 7, 148])))
        w = 16 // int(rng.choice([1, 3, 4, 16]))  # windows of one Q tile
        check(plan, n, L, w, int(rng.integers(1, 9)), int(rng.choice([1, 2, 7, 148])), tile=w)


def test_nothing_to_do(plan):
    for n in ([0], [0, 0, 0]):
        rows, _ = run(plan, n, [5] * len(n), 64, 4, 148)
        assert len(rows) == 0


def test_positions_past_32_bits(plan):
    # a sum of lengths beyond 2^31: the walk of the last ranges still ends at the last unit
    rows, cuts = run(plan, [1] * 8, [1 << 30] * 8, 64, 8, 148)
    assert cuts[0].total > 1 << 35
    last = rows[-1]
    assert (last[1], last[2], last[3]) == (7, 0, 7) and last[5] == last[6] == (1 << 30) // 128
    assert int((rows[:, 5] - rows[:, 4]).astype(np.int64).sum()) == 64 * ((1 << 30) // 128)


def test_cost_of_the_key_tiles_of_a_second_pass(plan):
    plan.keys_cost.restype = C.c_int64
    plan.keys_cost.argtypes = [C.c_int, C.c_int, C.c_int, C.c_int64]
    plan.keys_at.argtypes = [C.c_int] * 4 + [C.c_int64]
    rng = np.random.default_rng(6)
    for _ in range(300):
        tq = 128 // int(rng.choice([1, 2, 3, 5, 7, 8, 64, 128]))
        n = int(rng.integers(1, rng.choice([2, 40, 900])))
        L = max(1, n + int(rng.integers(-5, rng.choice([1, 200, 4000]))))
        tiles = -(-L // 128)
        cost = [(-(-n // tq) + 2) * tq - max(128 * j - (L - n), 0) for j in range(tiles)]
        assert min(cost) > 0
        ends = np.concatenate([[0], np.cumsum(cost)])
        assert [plan.keys_cost(n, L, tq, j) for j in range(tiles + 1)] == ends.tolist()
        for x in rng.integers(0, int(ends[-1]) + 2, 20).tolist() + ends.tolist():
            assert plan.keys_at(n, L, tq, tiles, x) == min(int(np.searchsorted(ends, x)), tiles)
    # past 32 bits
    n = L = 1 << 24
    tiles = n // 128
    assert plan.keys_cost(n, L, 32, tiles) == tiles * (n + 64) - 64 * tiles * (tiles - 1)


def test_warpgroups_that_share_a_key_tile(plan):
    for tiles in (1, 2, 3, 4):
        for q in range(1, 9):
            s = plan.sharers(tiles, q)
            assert 1 <= s <= q and s * tiles <= 4 and (s == q or (s + 1) * tiles > 4)
