"""The paged key/value cache on the GPU, further cases: lengths, tables, workspaces and sums that the cases of
test_gpu_paged.py do not reach.  Tolerances as derived there."""

import numpy as np
import pytest
import torch

import test_gpu_paged as T
from oracle import paged as P

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import token_skipping_sparse_b200 as S

I32 = torch.int32


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("each", [None, True, False])
def test_many_windows_whose_first_rows_see_no_slot(each, wide):
    # 50 new tokens over 10 cached: of a window's two Q tiles only the second one sees a slot, one window after another
    c = T.Cache([10] * 64, 16, 8, 128, seed=71)
    if wide:
        T.widen(c)
    T.check_attention(c, [50] * 64, 32, 8, 128, seed=72, each=each)
    T.check_attention(c, [50] * 64, 32, 8, 128, seed=72, each=each, lse=False)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d", [(28, 4, 64), (8, 8, 128)])
def test_windows_whose_first_rows_see_no_slot_among_others(Hq, Hkv, d, wide):
    new = [(7 * i * i + 3) % 150 for i in range(50)]
    lens = [max(0, n - (11 * i) % 170) + (200 if i % 5 == 0 else 0) for i, n in enumerate(new)]
    assert any(n > k > 0 for n, k in zip(new, lens))
    c = T.Cache(lens, 32, Hkv, d, seed=73)
    if wide:
        T.widen(c)
    T.check_attention(c, new, Hq, Hkv, d, seed=74)


def test_more_new_tokens_than_cached_ones_in_head_groups():
    # 6000 rows that see nothing before 20003 that do, the heads in groups; against the run of those 20003 alone
    none, L, Hq, Hkv, d, page = 6000, 20003, 32, 8, 128, 64
    g = torch.Generator(device="cuda").manual_seed(75)
    n_pages = -(-L // page)
    k, v = (torch.randn(n_pages, page, Hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = (torch.randn(none + L, Hq, d, generator=g, device="cuda") * 2).bfloat16()
    table = torch.arange(n_pages, dtype=I32, device="cuda")[None]
    o, e = S.spts_paged_attention(q, k, v, table, T.i32([L]), T.i32([0, none + L]), lse=True)
    S.check_device_status()
    assert not o[:none].any() and bool(torch.isneginf(e[:none]).all())
    want, ref = S.spts_paged_attention(q[none:], k, v, table, T.i32([L]), T.i32([0, L]), lse=True)
    S.check_device_status()
    # both are within a bound of the truth, so twice that apart; |q . k| <= |q| |k|, sum p |v| <= max |v|
    err = (d + 4) * 2.0 ** -23 * float(q.float().norm(dim=-1).max() * k.float().norm(dim=-1).max()) * d ** -0.5
    assert bool(((e[none:] - ref).abs() <= 2 * (err + 2.0 ** -21 * (1 + ref.abs()))).all())
    bound = 2 * (2 * T.U + 2 * err + 2.5e-4) * float(v.float().abs().max())
    assert bool(((o[none:].float() - want.float()).abs() <= bound).all())


def test_two_streams_without_workspaces_of_the_callers():
    # the same calls on two streams at once: attention in pieces, weights, eviction with the slots it keeps in between
    cs = [T.Cache([1500 + 300 * i, 900], 16, 8, 128, seed=76 + i, spare=80) for i in range(2)]
    qs = [T.packed([1 + 60 * i, 3], 32, 128, 78 + i) for i in range(2)]
    cus = [T.i32(cu) for cu, _ in qs]
    dst = [T.i32([c.free[:40], c.free[40:80]]) for c in cs]

    def once(i):
        w = torch.zeros(2, 8, cs[i].table.shape[1] * 16, device="cuda")
        o = S.spts_paged_attention(qs[i][1], *cs[i].args(), cus[i], weights=w)
        return (o, w) + S.spts_cache_evict(*cs[i].args(), w, 600, sink=4, recent=50, dst_table=dst[i], kept=True,
                                           weights_out=torch.empty(2, 8, 640, device="cuda"))

    ref = [once(i) for i in range(2)]
    S.check_device_status()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(12):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(once(i))
    torch.cuda.synchronize()
    S.check_device_status()
    for i in range(2):
        assert all(torch.equal(x, y) for out in outs[i] for x, y in zip(out, ref[i]))


def test_flags_of_calls_on_another_stream_are_found():
    c = T.Cache([20], 16, 2, 64, seed=80)
    cu, q = T.packed([1], 4, 64, 81)
    bad, cu = T.i32([10 ** 6]), T.i32(cu)
    S.check_device_status()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        S.spts_paged_attention(q, c.k, c.v, c.table, bad, cu)
    side.synchronize()
    with pytest.raises(S.SptsError):
        S.check_device_status()
    S.check_device_status()


@pytest.mark.parametrize("each", [True, False])
def test_evict_to_a_table_just_wide_enough_for_the_lengths(each):
    # every sequence is shorter than the budget, and so is a row of the destination
    lens, Hkv, d, page, keep = [1000, 17, 300], 2, 64, 16, 2048
    c = T.Cache(lens, page, Hkv, d, seed=82, spare=200)
    T.widen(c, 8192)
    w = T.weights_of(c, Hkv if each else 1, 83, "spread")
    dst = [[c.free.pop() if i * page < n else -1 for i in range(63)] for n in lens]
    want = P.cache_evict(c.np_k, c.np_v, c.rows, lens, T.f64(w), keep, 4, 100, dst, keep)
    new_lens, w_out, kept = S.spts_cache_evict(*c.args(), w, keep, sink=4, recent=100, dst_table=T.i32(dst), kept=True)
    S.check_device_status()
    assert new_lens.tolist() == lens and np.array_equal(kept.cpu().numpy(), want[4])
    assert np.array_equal(T.f64(w_out), want[2])
    assert np.array_equal(T.f64(c.k), want[0], equal_nan=True) and np.array_equal(T.f64(c.v), want[1], equal_nan=True)


@pytest.mark.parametrize("lens", [[300], [300, 41]])
def test_evict_to_the_first_columns_of_the_own_table(lens):
    # a view of the page table starts where the table does: the rows move in place, the weights to a row of their own
    page, keep = 16, 60
    c = T.Cache(lens, page, 2, 64, seed=84)
    w = T.weights_of(c, 2, 85, "spread")
    view = c.table[:, :4]
    want = P.cache_evict(c.np_k, c.np_v, c.rows, lens, T.f64(w), keep, 2, 9, c.rows, 64)
    new_lens, w_out, kept = S.spts_cache_evict(*c.args(), w, keep, sink=2, recent=9, dst_table=view, kept=True)
    S.check_device_status()
    assert new_lens.tolist() == want[3] and np.array_equal(kept.cpu().numpy(), want[4])
    assert np.array_equal(T.f64(w_out), want[2])
    for b, n in enumerate(want[3]):
        p, r = P.slot_rows(c.rows[b], n, page)
        assert np.array_equal(T.f64(c.k)[p, r], want[0][p, r]) and np.array_equal(T.f64(c.v)[p, r], want[1][p, r])


def check_long_sums(B, n, Hq, Hkv, d, each, width=None):
    """n new tokens of the first of B sequences, nothing else cached; K is 0 at the first ten slots and far off at all
    others, so that row i gives 1 / min(i + 1, 10) to each of the first min(i + 1, 10) slots, for every head.

    The scores are 0, or below the exponential's range.  Each weight is off by 2^-19 of itself (exp2, normaliser: the
    same for all rows), and the sum of a slot's by what is rounded outside of the compensated sum: 32 additions inside
    a block of rows, 2 more and 2 of the compensation, 3 for the shares of four warps, Hkv over the heads and one for
    what was there: not by their number.
    """
    page = 128
    n_pages = -(-n // page)
    k = torch.full((n_pages, page, Hkv, d), -16.0, dtype=torch.bfloat16, device="cuda")
    k.view(-1, Hkv, d)[:10] = 0
    v = torch.randn(n_pages, page, Hkv, d, device="cuda").bfloat16()
    q = torch.ones(n, Hq, d, dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, width or n_pages), -1, dtype=I32, device="cuda")
    table[0, :n_pages] = torch.arange(n_pages)
    w = torch.zeros(B, Hkv if each else 1, table.shape[1] * page, device="cuda")
    cu = [0] + [n] * B
    S.spts_paged_attention(q, k, v, table, T.i32([n] + [0] * (B - 1)), T.i32(cu), weights=w)
    S.check_device_status()
    rows = 1 / np.minimum(np.arange(n) + 1.0, 10)
    want = np.array([rows[j:].sum() for j in range(10)]) * (Hq // Hkv if each else Hq)
    got = T.f64(w[0])
    bound = (2.0 ** -19 + (32 + 2 + 2 + 3 + Hkv + 1) * 2.0 ** -24) * want
    assert np.all(np.abs(got[:, :10] - want) <= bound), np.abs(got[:, :10] / want - 1).max()
    assert not got[:, 10:].any() and not w[1:].any()


@pytest.mark.parametrize("each,width", [(True, None), (False, None), (False, 16500)])
def test_weights_of_many_rows_are_sums_of_all_of_them(each, width):
    # a wide table (16500 x 128 slots x 8 heads of fp32: above the room for sums per head): a unit walks all heads itself
    check_long_sums(1, 8192, 32, 8, 64, each, width)


@pytest.mark.parametrize("B", [256, 1024])
@pytest.mark.parametrize("each", [True, False])
def test_stored_weights_of_many_rows_are_sums_of_all_of_them(each, B):
    # few rows per sequence on average, all of them one sequence's: the attention leaves the scores (134 MB)
    check_long_sums(B, 1024, 32, 8, 128, each)


STEPS = {
    # new tokens of each sequence, earlier ones; one token each or less on average
    "steps": ([1] * 9, [0, 1, 15, 16, 127, 128, 300, 129, 511]),
    "some without a token": ([1, 0, 1, 0, 1, 1], [40, 200, 130, 0, 0, 255]),
    "one with several": ([5, 0, 0, 1, 0, 0, 1, 0], [130, 9, 0, 260, 40, 3, 0, 0]),
}


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("name", STEPS)
@pytest.mark.parametrize("G,Hkv,d", [(3, 2, 128), (5, 2, 64), (7, 1, 128), (7, 2, 64), (8, 2, 128), (16, 1, 128),
                                     (16, 2, 64)])
def test_steps_of_every_group_width(G, Hkv, d, name, wide):
    # Q tiles of 16 rows with and without padding rows, windows of one token (8 and 16 heads to a group) and of more
    new, old = STEPS[name]
    c = T.Cache([n + o for n, o in zip(new, old)], 16, Hkv, d, seed=90 + G)
    if wide:
        T.widen(c)
    T.check_attention(c, new, G * Hkv, Hkv, d, seed=91, lse=False)
    T.check_attention(c, new, G * Hkv, Hkv, d, seed=92)
    for each in (True, False):
        T.check_attention(c, new, G * Hkv, Hkv, d, seed=93, each=each)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("G,Hkv,d", [(1, 2, 128), (2, 2, 64), (3, 2, 128), (3, 1, 64), (5, 1, 128), (7, 2, 64)])
def test_few_rows_of_every_group_width(G, Hkv, d, wide):
    # up to 16 rows of a KV head per sequence on average: one to three tokens, and one sequence with more than a Q tile
    many = 128 // G + 3
    few = [1, 2, 3, 1] * 40
    count = next(k for k in range(2, 160) if (many + sum(few[:k])) * G <= 16 * (k + 1) and many + sum(few[:k]) > k + 1)
    new = [many] + few[:count]
    assert sum(new) > len(new) and sum(new) * G <= 16 * len(new)
    lens = [n + (37 * i) % 290 for i, n in enumerate(new)]
    c = T.Cache(lens, 32, Hkv, d, seed=94 + G)
    if wide:
        T.widen(c)
    T.check_attention(c, new, G * Hkv, Hkv, d, seed=95, lse=False)
    for each in (True, False):
        T.check_attention(c, new, G * Hkv, Hkv, d, seed=96, each=each)
