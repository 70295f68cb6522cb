"""The paged key/value cache on the GPU against its fp64 oracle: append, attention (with lse and accumulated
weights), eviction, and a run of them.

Tolerances are bounds, not fits.  With u = 2^-8 (half a bf16 step, relative):
  o        the weights p are rounded to bf16 for the product with V (u each) and the output once (u |o|); a score is
           off by at most e = (d + 4) 2^-23 aqk (fp32 accumulation of d products, aqk = scale sum |q k|), which moves
           every p by a factor of at most 1 + 2e; part of the exponentials is a polynomial with relative error
           1.1e-4, in p and in its normaliser:  |err| <= (u + 2e + 2.5e-4) sum p |v| + u |o|.
  lse      |err| <= e + 2^-21 (1 + |lse|): the score's error, and a few fp32 roundings (no polynomial here).
  weights  a call adds R weights p to a slot, each off by 2e + 2^-19 (exp2, normaliser) relative, summed in fp32:
           |err| <= (2e + 2^-19 + R 2^-24) added + 2^-23 (|before| + added).
  append   K: u |k'| and the angle's 2e-6 (|lo| + |hi|); V and every other slot: bit for bit.
  evict    bit for bit.
"""

import numpy as np
import pytest
import torch

from oracle import paged as P

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import token_skipping_sparse_b200 as S

U = 2.0 ** -8
I32 = torch.int32


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(v):
    return torch.tensor(v, dtype=I32, device="cuda")


class Cache:
    """Pages of random rows with NaN in every slot that holds no token."""

    def __init__(self, lens, page, Hkv, d, seed, spare=2, together=False, sizes=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        sizes = lens if sizes is None else sizes
        width = max(1, max(-(-n // page) for n in sizes))
        n_pages = sum(-(-n // page) for n in sizes) + spare
        free = [int(x) for x in rng.permutation(n_pages)]
        self.rows = [[free.pop() if i * page < n else -1 for i in range(width)] for n in sizes]
        self.free, self.lens, self.page = free, list(lens), page
        both = torch.randn(n_pages, 2, page, Hkv, d, generator=g).bfloat16()
        holds = torch.zeros(n_pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            p, r = P.slot_rows(self.rows[b], n, page)
            holds[p, r] = True
        both[~holds[:, None].expand(n_pages, 2, page)] = float("nan")
        self.np_k, self.np_v = f64(both[:, 0]), f64(both[:, 1])
        both = both.cuda()
        if together:  # K and V of a page side by side
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = both[:, 0].contiguous(), both[:, 1].contiguous()
        self.table, self.seq_lens = i32(self.rows), i32(lens)

    def args(self):
        return self.k, self.v, self.table, self.seq_lens


def packed(new, Hq, d, seed, pad=0, stride=0, gain=2.0):
    """cu and q [T, Hq, d]; `stride`: extra columns between rows, `pad`: rows behind the last sequence."""
    g = torch.Generator().manual_seed(seed + 77)
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    T = cu[-1] + pad
    q = (torch.randn(T, Hq * d + stride, generator=g) * gain).bfloat16().cuda()[:, :Hq * d].unflatten(1, (Hq, d))
    return cu, q


def check_attention(c, new, Hq, Hkv, d, seed, scale=None, each=None, lse=True, pad=0, stride=0, ws=None):
    cu, q = packed(new, Hq, d, seed, pad, stride)
    T = cu[-1]
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    hs = None if each is None else Hkv if each else 1
    w = before = None
    if hs:
        w = torch.rand(len(new), hs, c.table.shape[1] * c.page, generator=torch.Generator().manual_seed(seed)).cuda()
        before = f64(w)
    want = P.paged_attention(f64(q), c.np_k, c.np_v, c.rows, c.lens, cu, scale, hs)
    got = S.spts_paged_attention(q, *c.args(), i32(cu), scale=scale, out=out, lse=lse, weights=w, ws=ws)
    S.check_device_status(ws)
    o, e = got if lse else (got, None)
    assert o is out and torch.all(o[T:] == 7.0), "rows behind the last sequence"
    err = (d + 4) * 2.0 ** -23 * want["aqk"]
    diff = np.abs(f64(o)[:T] - want["o"][:T])
    bound = (U + 2 * err[:T, :, None] + 2.5e-4) * want["av"][:T] + U * np.abs(want["o"][:T])
    assert np.all(diff <= bound), ("o", np.nanmax(diff / (bound + 1e-30)))
    if lse:
        x, y = f64(e)[:T], want["lse"][:T]
        none = np.isneginf(y)
        assert np.array_equal(none, np.isneginf(x))
        bound = err[:T] + 2.0 ** -21 * (1 + np.abs(np.where(none, 0, y)))
        assert np.all(np.abs(np.where(none, 0, x) - np.where(none, 0, y)) <= bound)
    if hs:
        added, x = np.zeros_like(before), f64(w)
        n = min(want["weights"].shape[2], before.shape[2])
        added[..., :n] = want["weights"][..., :n]
        terms = max(new) * (Hq // hs)
        bound = (2 * err.max(initial=0) + 2.0 ** -19 + terms * 2.0 ** -24) * added + 2.0 ** -23 * (before + added)
        diff = np.abs(x - before - added)
        assert np.all(diff <= bound), ("weights", np.nanmax(diff / (bound + 1e-30)))
        for b, length in enumerate(c.lens):
            assert np.array_equal(x[b, :, length:], before[b, :, length:]), "weights behind the length"
    return q, cu


CASES = {
    # name: (new, old, Hq, Hkv, d, page)
    "one token, one slot": ([1], [0], 4, 1, 128, 16),
    "one token": ([1], [516], 8, 2, 128, 16),
    "steps": ([1] * 7, [0, 1, 15, 16, 127, 300, 129], 32, 8, 128, 16),
    "steps, narrow heads": ([1] * 5, [3, 64, 255, 256, 640], 16, 4, 64, 32),
    "steps, one head": ([1, 1], [77, 400], 1, 1, 128, 64),
    "few tokens each": ([2, 5, 3, 8], [130, 0, 511, 40], 8, 2, 128, 16),
    "whole prompts": ([129, 1, 64, 255], [0, 0, 0, 0], 8, 2, 128, 64),
    "whole prompts, narrow": ([200, 33], [0, 0], 4, 2, 64, 128),
    "chunks": ([70, 100], [300, 129], 8, 2, 128, 32),
    "chunks over large pages": ([90, 31], [500, 250], 4, 4, 128, 256),
    "mixed": ([1, 40, 0, 7, 1, 90], [200, 60, 33, 0, 0, 128], 14, 2, 64, 32),
    "three heads to a group": ([50, 1], [100, 260], 6, 2, 128, 16),
    "five heads to a group": ([30, 26], [0, 130], 5, 1, 128, 16),
    "sixteen heads to a group": ([20, 1, 9], [200, 90, 0], 16, 1, 64, 16),
    "all heads on one": ([3, 1], [140, 20], 64, 1, 128, 16),
    "a group as wide as a tile": ([3, 2], [30, 129], 128, 1, 64, 16),
    "nothing new": ([0, 0, 1], [40, 0, 10], 4, 2, 128, 16),
    "no sequence has anything": ([0, 0], [0, 0], 4, 2, 128, 16),
    "steps beside chunks": ([1] * 24 + [30, 40], [9 * i for i in range(24)] + [200, 70], 8, 2, 128, 16),
    "as many sequences as there may be": ([1, 0, 2, 1] * 256, [i % 19 for i in range(1024)], 4, 2, 64, 16),
    "many short ones": ([1, 2, 0, 3] * 12, [i % 37 for i in range(48)], 4, 2, 64, 16),
}


def widen(c, slots=1025):
    """A table row with room for more slots than units are dealt out whole for: the work is cut across CTAs."""
    more = -(-slots // c.page) - c.table.shape[1]
    if more > 0:
        c.table = torch.cat((c.table, torch.full((len(c.lens), more), -1, dtype=I32, device="cuda")), 1)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("name", CASES)
def test_attention(name, wide):
    new, old, Hq, Hkv, d, page = CASES[name]
    c = Cache([n + o for n, o in zip(new, old)], page, Hkv, d, seed=len(name))
    if wide:
        widen(c)
    check_attention(c, new, Hq, Hkv, d, seed=3, lse=False)
    check_attention(c, new, Hq, Hkv, d, seed=4)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("each", [True, False])
@pytest.mark.parametrize("name", CASES)
def test_attention_with_weights(name, each, wide):
    new, old, Hq, Hkv, d, page = CASES[name]
    c = Cache([n + o for n, o in zip(new, old)], page, Hkv, d, seed=len(name))
    if wide:
        widen(c)
    check_attention(c, new, Hq, Hkv, d, seed=5, each=each, lse=False)


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 4, 64)])
def test_attention_rows_that_see_no_slot_are_zero(Hq, Hkv, d):
    # more new tokens than cached ones: the first rows of the sequence come before its first slot
    c = Cache([5, 200, 0], 16, Hkv, d, seed=8)
    check_attention(c, [9, 330, 3], Hq, Hkv, d, seed=9, each=True)
    widen(c)
    check_attention(c, [9, 330, 3], Hq, Hkv, d, seed=9, each=True)
    check_attention(c, [0, 1, 1], Hq, Hkv, d, seed=9, each=True)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_strides_padding_and_scale(d):
    c = Cache([300, 17, 90], 16, 2, d, seed=10, together=True)
    check_attention(c, [40, 1, 3], 8, 2, d, seed=11, scale=0.3, pad=5, stride=24, each=False)
    wide = torch.full((3, 60), 10 ** 6, dtype=I32, device="cuda")  # entries past a row's pages are not read
    wide[:, :c.table.shape[1]] = torch.where(c.table < 0, -5, c.table)
    c.table = wide[:, :c.table.shape[1] + 3]
    check_attention(c, [40, 1, 3], 8, 2, d, seed=12)


def test_attention_over_shared_pages():
    # two sequences with the same first pages, and one that names a page twice
    c = Cache([64, 64, 48], 16, 2, 128, seed=13)
    c.rows[1][:3] = c.rows[0][:3]
    c.rows[2][2] = c.rows[2][0]
    c.table = i32(c.rows)
    check_attention(c, [5, 1, 2], 8, 2, 128, seed=14, each=True)


@pytest.mark.parametrize("gain", [0.0, 40.0])
def test_attention_flat_and_sharp_scores(gain):
    c = Cache([700, 65], 32, 2, 128, seed=15)
    cu, q = packed([33, 1], 8, 128, 16, gain=gain)
    o, e = S.spts_paged_attention(q, *c.args(), i32(cu), lse=True)
    want = P.paged_attention(f64(q), c.np_k, c.np_v, c.rows, c.lens, cu)
    err = 132 * 2.0 ** -23 * want["aqk"]
    assert np.all(np.abs(f64(o) - want["o"]) <= (U + 2 * err[..., None] + 2.5e-4) * want["av"] + U * np.abs(want["o"]))
    assert np.all(np.abs(f64(e) - want["lse"]) <= err + 2.0 ** -21 * (1 + np.abs(want["lse"])))


@pytest.mark.parametrize("each", [True, False])
def test_attention_long_enough_for_head_groups(each):
    # K and V of 82 MB shared by 19 windows of new tokens: the heads are taken in groups.  fp64 on the GPU, head by head
    n, L, Hq, Hkv, d, page = 1201, 20003, 32, 8, 128, 64
    g = torch.Generator(device="cuda").manual_seed(41)
    n_pages = -(-L // page)
    k, v = (torch.randn(n_pages, page, Hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    k.view(-1, Hkv, d)[L:], v.view(-1, Hkv, d)[L:] = float("nan"), float("nan")
    q = (torch.randn(n, Hq, d, generator=g, device="cuda") * 2).bfloat16()
    table = torch.arange(n_pages, dtype=I32, device="cuda")[None]
    w = torch.zeros(1, Hkv if each else 1, n_pages * page, device="cuda")
    o, e = S.spts_paged_attention(q, k, v, table, i32([L]), i32([0, n]), lse=True, weights=w)
    S.check_device_status()
    sees = torch.arange(L, device="cuda") <= L - n + torch.arange(n, device="cuda")[:, None]
    want_w = torch.zeros(w.shape, dtype=torch.float64, device="cuda")
    for h in range(Hq):
        K, V = (x.view(-1, Hkv, d)[:L, h // (Hq // Hkv)].double() for x in (k, v))
        s = (q[:, h].double() @ K.T * d ** -0.5).masked_fill(~sees, -np.inf)
        err = (d + 4) * 2.0 ** -23 * float((q[:, h].double().abs() @ K.abs().T).max()) * d ** -0.5
        a = s.softmax(-1)
        bound = (U + 2 * err + 2.5e-4) * (a @ V.abs()) + U * (a @ V).abs()
        assert bool(((o[:, h].double() - a @ V).abs() <= bound).all()), h
        ref = s.logsumexp(-1)
        assert bool(((e[:, h].double() - ref).abs() <= err + 2.0 ** -21 * (1 + ref.abs())).all())
        want_w[0, h // (Hq // Hkv) if each else 0, :L] += a.sum(0)
    bound = (2 * err + 2.0 ** -19 + n * (Hq // w.shape[1]) * 2.0 ** -24) * want_w
    assert bool(((w.double() - want_w).abs() <= bound).all())


@pytest.mark.parametrize("wide", [False, True])
def test_one_sequence_does_not_reach_another(wide):
    # non-finite rows of one sequence, and of its neighbour in the packed rows
    c = Cache([100, 50, 70], 16, 2, 128, seed=17)
    if wide:
        widen(c)
    p, r = P.slot_rows(c.rows[1], 50, 16)
    cu, q = packed([60, 20, 1], 8, 128, 18)
    clean = S.spts_paged_attention(q, *c.args(), i32(cu))
    c.k[p, r], c.v[p, r] = float("nan"), float("inf")
    q[60:80] = float("nan")
    o = S.spts_paged_attention(q, *c.args(), i32(cu))
    assert torch.equal(o[:60], clean[:60]) and torch.equal(o[80:], clean[80:])
    assert torch.all(torch.isnan(o[60:80]))


def test_attention_twice_gives_the_same_bits():
    c = Cache([900, 1500, 31], 16, 8, 128, seed=19)
    cu, q = packed([1, 130, 2], 32, 128, 20)
    runs = []
    for _ in range(3):
        w = torch.zeros(3, 8, c.table.shape[1] * 16, device="cuda")
        o, e = S.spts_paged_attention(q, *c.args(), i32(cu), lse=True, weights=w)
        runs.append((o, e, w))
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(r, runs[0]))


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("rope", [True, False])
@pytest.mark.parametrize("new,old,Hkv,d,page", [([1], [0], 1, 64, 16), ([1] * 5, [0, 15, 16, 100, 31], 8, 128, 16),
                                                ([200, 0, 33], [0, 20, 500], 2, 128, 64),
                                                ([3, 130], [255, 126], 3, 64, 128), ([300], [10], 5, 128, 256)])
def test_append(new, old, Hkv, d, page, rope):
    lens = [n + o for n, o in zip(new, old)]
    c = Cache(old, page, Hkv, d, seed=21, sizes=lens)
    cu, both = packed(new, 2 * Hkv, d, 22, pad=3, gain=1.0)
    k, v = both[:, :Hkv], both[:, Hkv:]
    pos = None
    if rope:
        pos = np.concatenate([np.arange(n) * 3 + o * 5 + (10 ** 7 if b == 0 else 0)
                              for b, (n, o) in enumerate(zip(new, old))] + [np.arange(3)])
    want_k, want_v = P.cache_append(f64(k), f64(v), c.np_k, c.np_v, c.rows, lens, cu, pos)
    S.spts_cache_append(k, v, c.k, c.v, c.table, i32(lens), i32(cu), None if pos is None else i32(pos.tolist()))
    S.check_device_status()
    got_k, got_v = f64(c.k), f64(c.v)
    assert np.array_equal(got_v, want_v, equal_nan=True)
    if not rope:
        assert np.array_equal(got_k, want_k, equal_nan=True)
        return
    touched = ~np.isnan(want_k) & (np.isnan(c.np_k) | (want_k != c.np_k))
    same = ~touched
    assert np.array_equal(got_k[same], want_k[same], equal_nan=True)
    half = np.abs(want_k[..., :d // 2]) + np.abs(want_k[..., d // 2:])
    bound = U * np.abs(want_k) + 2e-6 * np.sqrt(2) * np.concatenate((half, half), -1)
    assert np.all(np.abs(got_k - want_k)[touched] <= bound[touched])


# ------------------------------------------------------------------ evict
def weights_of(c, Hs, seed, kind):
    g = torch.Generator().manual_seed(seed)
    n = c.table.shape[1] * c.page
    if kind == "ties":
        w = torch.randint(-2, 3, (len(c.lens), Hs, n), generator=g).float() * 0.5
        w[w == 0] = -0.0
        w[..., ::3] = w[..., ::3].abs()
    elif kind == "equal":
        w = torch.full((len(c.lens), Hs, n), 0.25)
    else:
        w = torch.rand(len(c.lens), Hs, n, generator=g) ** 4
    for b, length in enumerate(c.lens):
        w[b, :, length:] = float("nan")  # nothing of this may count
    return w.cuda()


@pytest.mark.parametrize("kind", ["spread", "ties", "equal"])
@pytest.mark.parametrize("lens,Hkv,d,page,keep,sink,recent,each", [
    ([40], 1, 64, 16, 1, 0, 0, True), ([300, 7, 0, 64, 65], 2, 128, 16, 64, 4, 16, True),
    ([300, 7, 0, 64, 65], 2, 128, 16, 64, 4, 16, False), ([500, 513], 3, 64, 32, 100, 0, 100, True),
    ([500, 90], 2, 128, 128, 200, 200, 0, False), ([2500, 1200, 4100], 8, 128, 64, 1030, 1, 31, True),
    ([5000], 2, 64, 16, 4999, 0, 0, False), ([33, 20], 2, 64, 16, 1000, 3, 5, True),
])
def test_evict(lens, Hkv, d, page, keep, sink, recent, each, kind):
    kept_lens = [min(n, keep) for n in lens]
    Hs = Hkv if each else 1
    c = Cache(lens, page, Hkv, d, seed=23, spare=sum(-(-n // page) for n in kept_lens) + 1, together=True)
    w = weights_of(c, Hs, 24, kind)
    width = max(1, max(-(-n // page) for n in kept_lens))
    dst = [[c.free.pop() if i * page < n else -1 for i in range(width)] for n in kept_lens]
    # to other pages
    need = min(keep, c.table.shape[1] * page)
    out_width = max(width * page, need)
    want = P.cache_evict(c.np_k, c.np_v, c.rows, lens, f64(w), keep, sink, recent, dst, out_width)
    k0, v0, w0 = c.k.clone(), c.v.clone(), w.clone()
    w_out = torch.full((len(lens), Hs, out_width), 9.0, device="cuda")
    new_lens, got_w, kept = S.spts_cache_evict(*c.args(), w, keep, sink, recent, dst_table=i32(dst), weights_out=w_out,
                                               kept=True)
    S.check_device_status()
    assert got_w is w_out and new_lens.tolist() == want[3]
    assert np.array_equal(kept.cpu().numpy(), want[4])
    assert np.array_equal(f64(w_out), want[2]) and torch.equal(w.view(I32), w0.view(I32))
    assert np.array_equal(f64(c.k), want[0], equal_nan=True) and np.array_equal(f64(c.v), want[1], equal_nan=True)
    # in place, lengths too
    c.k.copy_(k0)
    c.v.copy_(v0)
    want = P.cache_evict(c.np_k, c.np_v, c.rows, lens, f64(w), keep, sink, recent, c.rows, w.shape[2])
    new_lens, got_w, kept = S.spts_cache_evict(*c.args(), w, keep, sink, recent, new_lens=c.seq_lens, kept=True)
    S.check_device_status()
    assert got_w is w and new_lens is c.seq_lens and c.seq_lens.tolist() == want[3]
    assert np.array_equal(kept.cpu().numpy(), want[4])
    for b, n in enumerate(want[3]):
        p, r = P.slot_rows(c.rows[b], n, page)
        assert np.array_equal(f64(c.k)[p, r], want[0][p, r]) and np.array_equal(f64(c.v)[p, r], want[1][p, r])
        assert np.array_equal(f64(w)[b], want[2][b])


def test_evict_flags_a_weight_that_is_not_finite():
    c = Cache([100, 60], 16, 1, 64, seed=25)
    w = weights_of(c, 1, 26, "spread")
    w[0, 0, 50] = float("inf")
    S.check_device_status()
    S.spts_cache_evict(*c.args(), w, 64)
    with pytest.raises(S.SptsError):
        S.check_device_status()


# ------------------------------------------------------------------ bad lengths, offsets and pages
@pytest.mark.parametrize("bad", ["length", "negative length", "page", "negative page", "offset", "descending"])
def test_bad_device_values_are_flagged_and_reach_no_other_sequence(bad):
    lens, new = [100, 50, 70], [60, 20, 1]
    c = Cache(lens, 16, 2, 128, seed=27)
    cu, q = packed(new, 8, 128, 28)
    want = P.paged_attention(f64(q), c.np_k, c.np_v, c.rows, lens, cu)
    S.check_device_status()
    widen(c)
    rows, sizes = c.table.tolist(), list(lens)
    if bad == "length":
        sizes[1] = 10 ** 9
    elif bad == "negative length":
        sizes[1] = -4
    elif bad == "page":
        rows[1][1] = c.k.shape[0]
    elif bad == "negative page":
        rows[1][0] = -1
    elif bad == "offset":
        cu[3] = 10 ** 6
    else:
        cu[2] = 10
    w = torch.zeros(3, 2, c.table.shape[1] * 16, device="cuda")
    o = S.spts_paged_attention(q, c.k, c.v, i32(rows), i32(sizes), i32(cu), weights=w)
    with pytest.raises(S.SptsError):
        S.check_device_status()
    # the other sequences are right within the bounds (their bits may move: the work is cut elsewhere)
    err = 132 * 2.0 ** -23 * want["aqk"][..., None]
    fine = np.abs(f64(o) - want["o"]) <= (U + 2 * err + 2.5e-4) * want["av"] + U * np.abs(want["o"])
    assert np.all(fine[:60]) or bad == "descending"
    assert np.all(fine[80:]) or bad in ("offset", "descending")


def test_bad_pages_and_missing_slots_are_flagged_by_append_and_evict():
    c = Cache([20, 10], 16, 2, 64, seed=29)
    cu, kv = packed([4, 12], 2, 64, 30)
    k0 = c.k.clone()
    S.check_device_status()
    S.spts_cache_append(kv, kv, *c.args(), i32(cu))  # 12 new tokens, 10 slots
    with pytest.raises(S.SptsError):
        S.check_device_status()
    p, r = P.slot_rows(c.rows[1], 10, 16)
    assert torch.equal(c.k[p, r], kv[6:16])
    rows = [list(x) for x in c.rows]
    rows[0][1] = 10 ** 6
    c.k.copy_(k0)
    S.spts_cache_append(kv[:4], kv[:4], c.k, c.v, i32(rows), i32([20, 10]), i32([0, 4, 4]))
    with pytest.raises(S.SptsError):
        S.check_device_status()
    assert torch.equal(c.k.view(torch.int16), k0.view(torch.int16))
    S.spts_cache_evict(c.k, c.v, i32(rows), c.seq_lens, torch.rand(2, 2, 32, device="cuda"), 8)
    with pytest.raises(S.SptsError):
        S.check_device_status()


def test_waits_that_run_out_end_the_call_with_a_status():
    # (large enough for waits that the barrier's own patience does not cover)
    c = Cache([4000, 90], 16, 8, 128, seed=42)
    cu, q = packed([2000, 1], 32, 128, 43)
    w = torch.zeros(2, 8, c.table.shape[1] * 16, device="cuda")
    clean = S.spts_paged_attention(q, *c.args(), i32(cu), weights=w.clone())
    S.check_device_status()
    limit = S.get_wait_limit_ns()
    S.set_wait_limit_ns(0)
    try:
        S.spts_paged_attention(q, *c.args(), i32(cu), weights=w.clone())
        with pytest.raises(S.SptsError, match="gave up"):
            S.check_device_status()
    finally:
        S.set_wait_limit_ns(limit)
    assert torch.equal(S.spts_paged_attention(q, *c.args(), i32(cu), weights=w), clean)
    S.check_device_status()


# ------------------------------------------------------------------ sizes
def test_pages_beyond_32_bit_offsets():
    # 2.2e9 elements of K and of V; the sequence's pages are the last ones
    page, Hkv, d, n_pages = 256, 8, 128, 8400
    k, v = (torch.empty(n_pages, page, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 31
    table = i32([[n_pages - 1, n_pages - 3, n_pages - 5]])
    L = 600
    cu, kv = packed([L], Hkv, d, 44, gain=1.0)
    _, q = packed([7], 8, d, 45)
    S.spts_cache_append(kv, kv * 0.5, k, v, table, i32([L]), i32([0, L]))
    o = S.spts_paged_attention(q, k, v, table, i32([L]), i32([0, 7]))
    small = [x[[n_pages - 1, n_pages - 3, n_pages - 5]].contiguous() for x in (k, v)]
    own = i32([[0, 1, 2]])
    assert torch.equal(small[0].view(-1, Hkv, d)[:L], kv)
    assert torch.equal(o, S.spts_paged_attention(q, *small, own, i32([L]), i32([0, 7])))
    w = torch.rand(1, Hkv, 3 * page, device="cuda")
    lens, w_out, kept = S.spts_cache_evict(k, v, table, i32([L]), w, 200, dst_table=i32([[n_pages - 2]]), kept=True)
    S.check_device_status()
    for g in range(Hkv):
        assert torch.equal(k[n_pages - 2, :200, g], kv[kept[0, g].long(), g])


def test_evict_of_rows_too_long_to_hold():
    # 410000 slots: a cluster's shared memory does not hold their keys
    page, d, L, keep = 256, 64, 410003, 1500
    n_pages = -(-L // page)
    k = torch.randn(n_pages + 6, page, 1, d, device="cuda").bfloat16()
    v = torch.randn(n_pages + 6, page, 1, d, device="cuda").bfloat16()
    w = torch.randint(0, 5000, (1, 1, n_pages * page), device="cuda").float()  # ties at the threshold
    table = torch.arange(n_pages, dtype=I32, device="cuda")[None]
    dst = torch.arange(n_pages, n_pages + 6, dtype=I32, device="cuda")[None]
    lens, w_out, kept = S.spts_cache_evict(k, v, table, i32([L]), w, keep, sink=3, recent=10, dst_table=dst, kept=True)
    S.check_device_status()
    x = w[0, 0, 3:L - 10].cpu().numpy()
    order = np.argsort(-x, kind="stable")[:keep - 13] + 3
    want = np.sort(np.concatenate((np.arange(3), order, np.arange(L - 10, L))))
    assert np.array_equal(kept[0, 0].cpu().numpy(), want) and lens.tolist() == [keep]
    idx = torch.from_numpy(want).cuda()
    assert torch.equal(w_out[0, 0, :keep], w[0, 0, idx]) and not w_out[0, 0, keep:].any()
    for x in (k, v):
        assert torch.equal(x[n_pages:].view(-1, d)[:keep], x.view(-1, d)[idx])


@pytest.mark.parametrize("new", [[1, 1], [40, 3]])
def test_weights_over_all_heads_with_a_wide_table(new):
    # a page table row for 2.2 M slots: neither scores nor partial sums per head have scratch
    c = Cache([300, 130], 16, 8, 64, seed=46)
    wide = torch.full((2, 140000), -1, dtype=I32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    check_attention(c, new, 16, 8, 64, seed=47, each=False)


@pytest.mark.parametrize("each", [True, False])
@pytest.mark.parametrize("B,Hq,Hkv,d", [(7, 64, 1, 128), (40, 128, 2, 64), (110, 128, 2, 64), (3, 1, 1, 128),
                                        (5, 128, 1, 128)])
def test_weights_of_few_and_many_key_tiles(B, Hq, Hkv, d, each):
    # few K tiles with many Q tiles each go round one by one, others by equal cost; one to four warpgroups to a tile
    lens = [1 + (37 * i * i + 131 * i) % 900 for i in range(B)]
    new = [min(1 + i % 9 if Hkv > 1 else 30 * (i + 1) if Hq > 1 else 300 * (i + 1), n) for i, n in enumerate(lens)]
    c = Cache(lens, 32, Hkv, d, seed=61)
    check_attention(c, new, Hq, Hkv, d, seed=62, each=each)


def test_weights_twice_give_the_same_bits():
    lens = [1 + (53 * i * i + 17 * i) % 700 for i in range(60)]
    new = [min(1 + 7 * (i % 30), n) for i, n in enumerate(lens)]
    c = Cache(lens, 64, 4, 128, seed=63)
    cu, q = packed(new, 16, 128, 64)
    runs = []
    for _ in range(4):
        w = torch.zeros(60, 1, c.table.shape[1] * 64, device="cuda")
        S.spts_paged_attention(q, *c.args(), i32(cu), weights=w)
        runs.append(w)
    assert all(torch.equal(w, runs[0]) for w in runs)
    # a row's weights add up to 1: each is off by 2 (d + 4) 2^-23 of the scores' absolute products (about 14), and 2^-19
    assert abs(float(runs[0].double().sum()) - 16 * sum(new)) < 1e-3 * 16 * sum(new)


# ------------------------------------------------------------------ streams, graphs, a run of all
def test_two_streams_with_workspaces_of_their_own():
    cs = [Cache([700 + 50 * i, 90], 16, 2, 128, seed=31 + i) for i in range(2)]
    qs = [packed([1 + 40 * i, 3], 8, 128, 33 + i) for i in range(2)]
    ref = [S.spts_paged_attention(q, *c.args(), i32(cu)) for c, (cu, q) in zip(cs, qs)]
    ws = [torch.zeros(S.spts_paged_attention_workspace(q, *c.args()), dtype=torch.uint8, device="cuda")
          for c, (_, q) in zip(cs, qs)]
    cus = [i32(cu) for cu, _ in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(8):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(S.spts_paged_attention(qs[i][1], *cs[i].args(), cus[i], ws=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        S.check_device_status(ws[i])
        assert all(torch.equal(o, ref[i]) for o in outs[i])


def decode(c, q, kv, pos, cu, w, keep, ws):
    """One step: the new tokens go into the cache, attend, and the cache is cut to its budget."""
    c.seq_lens += 1
    S.spts_cache_append(kv, kv * 0.5, *c.args(), cu, pos=pos, ws=ws)
    o = S.spts_paged_attention(q, *c.args(), cu, weights=w, ws=ws)
    S.spts_cache_evict(*c.args(), w, keep, sink=2, recent=8, new_lens=c.seq_lens, ws=ws)
    return o


def test_steps_of_decoding_under_a_budget_eager_and_captured():
    B, Hq, Hkv, d, keep, steps = 3, 8, 2, 128, 60, 6
    g = torch.Generator().manual_seed(35)
    q, kv = (torch.randn(steps, B, h, d, generator=g).bfloat16().cuda() for h in (Hq, Hkv))
    caches = [Cache([58, 20, 60], 16, Hkv, d, seed=36, sizes=[80, 80, 80]) for _ in range(2)]
    cu, pos = i32([0, 1, 2, 3]), i32([100, 200, 300])
    w = [torch.zeros(B, Hkv, 80, device="cuda") for _ in range(2)]
    need = max(S.spts_paged_attention_workspace(q[0], *caches[0].args(), weights=True),
               S.spts_cache_evict_workspace(*caches[0].args(), w[0], keep))
    ws = [torch.zeros(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    eager, c = [], caches[0]
    for i in range(steps):
        eager.append(decode(c, q[i], kv[i], pos, cu, w[0], keep, ws[0]))
    # the first step against the oracle, and the budget held
    ref = Cache([58, 20, 60], 16, Hkv, d, seed=36, sizes=[80, 80, 80])
    lens = [n + 1 for n in ref.lens]
    k1, v1 = P.cache_append(f64(kv[0]), f64(kv[0] * 0.5), ref.np_k, ref.np_v, ref.rows, lens, [0, 1, 2, 3],
                            [100, 200, 300])
    k1 = f64(torch.from_numpy(k1).bfloat16())
    want = P.paged_attention(f64(q[0]), k1, v1, ref.rows, lens, [0, 1, 2, 3], None, Hkv)
    assert np.all(np.abs(f64(eager[0]) - want["o"]) <= 2e-2)
    assert c.seq_lens.tolist() == [60, 26, 60]
    # captured once, replayed with new inputs in the same places
    c = caches[1]
    qs, kvs = q[0].clone(), kv[0].clone()
    decode_state = (c.k.clone(), c.v.clone(), c.seq_lens.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm up, then put the state back
        decode(c, qs, kvs, pos, cu, w[1], keep, ws[1])
        for t, s in zip((c.k, c.v, c.seq_lens), decode_state):
            t.copy_(s)
        w[1].zero_()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = decode(c, qs, kvs, pos, cu, w[1], keep, ws[1])
    for i in range(steps):
        qs.copy_(q[i])
        kvs.copy_(kv[i])
        graph.replay()
        assert torch.equal(o, eager[i]), i
    for x in ws:
        S.check_device_status(x)
    assert torch.equal(w[0], w[1]) and c.seq_lens.tolist() == [60, 26, 60]
    for a, b in ((caches[0].k, caches[1].k), (caches[0].v, caches[1].v)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_tensors_on_another_device_are_refused():
    c = Cache([20], 16, 2, 64, seed=48)
    cu, q = packed([1], 4, 64, 49)
    for args in ((c.k, c.v, c.table.cpu(), c.seq_lens), (c.k, c.v.cpu(), c.table, c.seq_lens)):
        with pytest.raises(ValueError):
            S.spts_paged_attention(q, *args, i32(cu))
    with pytest.raises(ValueError, match="cu_q"):
        S.spts_paged_attention(q, *c.args(), torch.tensor(cu, dtype=I32))
    with pytest.raises(ValueError, match="weights"):
        S.spts_paged_attention(q, *c.args(), i32(cu), weights=torch.zeros(1, 2, 16, device="cuda"))


def test_capture_needs_a_workspace_of_the_callers():
    c = Cache([20], 16, 2, 64, seed=37)
    cu, q = packed([1], 4, 64, 38)
    cu = i32(cu)
    S.spts_paged_attention(q, *c.args(), cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="ws"):
            S.spts_paged_attention(q, *c.args(), cu)


def test_a_prompt_in_parts_gives_what_the_whole_prompt_gives():
    # fed whole, in two uneven parts, and against the attention of the skipping prefill with every row selected
    n, Hq, Hkv, d, page = 333, 8, 2, 128, 32
    g = torch.Generator().manual_seed(39)
    q, k, v = (torch.randn(n, h, d, generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv))
    pos = torch.arange(n, dtype=I32, device="cuda")
    turned = S.spts_rope(k.clone(), pos)
    ref = f64(S.spts_reduced_attention(q, pos, turned, v, pos))
    for parts in ([333], [200, 133], [1, 331, 1]):
        c = Cache([0], page, Hkv, d, seed=40, sizes=[n])
        at, outs = 0, []
        for m in parts:
            c.seq_lens += m
            S.spts_cache_append(k[at:at + m], v[at:at + m], *c.args(), i32([0, m]), pos=pos[at:at + m])
            outs.append(S.spts_paged_attention(q[at:at + m], *c.args(), i32([0, m])))
            at += m
        S.check_device_status()
        p, r = P.slot_rows(c.rows[0], n, page)
        assert torch.equal(c.k[p, r], turned)
        assert np.abs(f64(torch.cat(outs)) - ref).max() <= 2e-2
