"""The order of the attention's warps over the paged cache: whatever the lengths, none of the two softmax warpgroups
gets ahead of the other and no wait skips a phase (CPU: the kernel's plan, compiled for the host, and a model of the
barriers that its MMA warp and its warpgroups meet at)."""

import ctypes as C
import itertools
import os
import shutil
import subprocess

import numpy as np
import pytest

import test_paged_plan as plan_tests

SHIM = plan_tests.SHIM + r"""
extern "C" int first_end(int n, int L, int w, int tile, int p, int t0, int t1) {
  return plan_first_end(PlanSeq{n, L}, PlanShape{w, tile}, p, t0, t1);
}
extern "C" int has_slot(int t, int max_pages, int page_shift) { return paged_has_slot(t, max_pages, page_shift); }
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    at = tmp_path_factory.mktemp("order")
    (at / "shim.cpp").write_text(SHIM)
    so = str(at / "order.so")
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", plan_tests.CSRC, str(at / "shim.cpp"), "-o", so],
                   check=True)
    return C.CDLL(so)


class Barrier:
    """An mbarrier: `count` arrivals complete a phase; a wait is for the completion of a phase of one parity."""

    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        return (self.phase & 1) != parity


def meet(items, order):
    """Runs the MMA warp and the two softmax warpgroups over `items` (two Q tiles?, key tiles, key tiles of the first Q
    tile), always the first of `order` that can go on; True if all three come to the end."""
    s_full, o_done = [Barrier(1), Barrier(1)], [Barrier(1), Barrier(1)]
    p_ready, o_free, x_full = [Barrier(1), Barrier(1)], Barrier(2), Barrier(2)
    arrived = [0, 0]

    def mma():
        used, units = [0, 0], 0
        for two, n, n_a in items:
            if n <= 0:
                continue
            tiles = [n_a, n] if two else [(n + 1) // 2, n // 2]
            first = True
            for x in (0, 1):
                if tiles[x]:
                    s_full[x].arrive()  # S of the first tile
            steps = [(i, x) for i in range(n) for x in (0, 1) if i < tiles[x]] if two else \
                [(i // 2, i % 2) for i in range(n)]
            for i, x in steps:
                if first:
                    first = False
                    yield lambda: o_free.passed((units & 1) ^ 1)
                yield lambda: p_ready[x].passed(used[x] & 1)
                used[x] += 1
                o_done[x].arrive()
                if i + 1 < tiles[x]:
                    s_full[x].arrive()
            units += 1

    def softmax(x):
        used, joins = 0, 0
        for two, n, n_a in items:
            own = (n if x else n_a) if two else (n + 1 - x) >> 1
            for _ in range(own):
                yield lambda: s_full[x].passed(used & 1)
                used += 1
                p_ready[x].arrive()
            if n <= 0:
                continue
            if own > 0:
                yield lambda: o_done[x].passed((used - 1) & 1)
            if not two:
                x_full.arrive()
                yield lambda: x_full.passed(joins & 1)
                joins += 1
            # both warpgroups have arrived for every unit but at most the last
            assert arrived[x] <= arrived[1 - x], "a warpgroup arrives twice in one phase"
            arrived[x] += 1
            o_free.arrive()

    agents = [mma(), softmax(0), softmax(1)]
    waits = [next(a, None) for a in agents]
    while any(waits):
        for k in order:
            if waits[k] is not None and waits[k]():
                waits[k] = next(agents[k], None)
                break
        else:
            return False
    return True


def items_of(plan, n, L, w, tile, heads, ctas, groups=1):
    """The pieces of each CTA, as its warps get them; `groups` head groups of `heads` heads alike."""
    rows, _ = plan_tests.run(plan, n, L, w, heads, ctas, tile)
    out = [[] for _ in range(ctas)]
    for r, b, p, _, t0, t1, _, whole, _ in rows.tolist():
        if t0 >= t1 and not whole:
            continue
        a_end = plan.first_end(n[b], L[b], w, tile, p, t0, t1)
        out[r].append((w > tile and n[b] - p * w > tile, t1 - t0, max(min(a_end, t1) - t0, 0)))
    return [x * groups for x in out]


def check(plan, n, L, w, tile, heads, ctas, groups=1):
    seen = set()
    for items in items_of(plan, n, L, w, tile, heads, ctas, groups):
        short = []  # the same with fewer tiles, of which the first Q tile misses as many
        for two, k, a in items[:24]:
            fewer = k if k < 6 else 6 + k % 2
            short.append((two, fewer, max(fewer - (k - a), min(a, 1)) if two else fewer))
        short = tuple(short)
        if short in seen:
            continue
        seen.add(short)
        for order in itertools.permutations(range(3)):
            assert meet(short, order), (n, L, short)


def test_the_model_sees_a_warpgroup_without_tiles():
    # the first Q tile of both units sees nothing and has no key tile: its warpgroup runs ahead
    with pytest.raises(AssertionError, match="twice"):
        for order in itertools.permutations(range(3)):
            assert meet([(True, 1, 0), (True, 1, 0), (True, 1, 0)], order)
    assert all(meet([(True, 1, 1), (True, 3, 2), (False, 1, 0), (True, 1, 1)], o) for o in itertools.permutations(range(3)))


@pytest.mark.parametrize("groups", [1, 4])
def test_more_new_tokens_than_cached_ones(plan, groups):
    for heads in (2, 8):
        check(plan, [50] * 64, [10] * 64, 64, 32, heads, 148, groups)
        check(plan, [9, 330, 3], [5, 200, 0], 64, 32, heads, 3, groups)
    check(plan, [3000], [200], 64, 32, 8, 148, groups)
    check(plan, [100000], [10000], 256, 128, 1, 148, groups)


@pytest.mark.parametrize("groups", [1, 2])
def test_ragged_batches(plan, groups):
    rng = np.random.default_rng(7)
    for _ in range(60):
        B = int(rng.integers(1, 30))
        n = [int(x) for x in rng.integers(0, rng.choice([2, 90, 300]), B)]
        L = [int(max(0, m + rng.integers(-m, rng.choice([1, 50, 900])))) for m in n]
        tile = 128 // int(rng.choice([1, 2, 3, 4, 7, 32]))
        check(plan, n, L, 2 * tile, tile, int(rng.integers(1, 5)), int(rng.choice([1, 2, 7, 148])), groups)


def test_every_warpgroup_has_a_tile_of_every_piece(plan):
    for n, L in ((50, 10), (330, 200), (500, 4000), (64, 64), (100, 0)):
        for p in range(-(-n // 64)):
            seen = max(L - n + min((p + 1) * 64, n), 0)
            first = max(L - n + min(p * 64 + 32, n), 0)
            tiles = -(-seen // 128)
            for t0, t1 in itertools.combinations(range(tiles + 1), 2):
                end = plan.first_end(n, L, 64, 32, p, t0, t1)
                assert t0 < end <= t1 and end >= min(-(-first // 128), t1)
            assert plan.first_end(n, L, 64, 32, p, tiles, tiles) == tiles


def test_only_slots_of_a_table_row_are_slots(plan):
    for shift in (4, 8):
        for pages in (1, 3, 1 << 18):
            cap = pages << shift
            for t, ok in ((0, 1), (cap - 1, 1), (cap, 0), (cap + 1, 0), (-1, 0), (2 ** 31 - 1, 0), (-2 ** 31, 0)):
                assert bool(plan.has_slot(t, pages, shift)) == bool(ok), (t, pages, shift)
