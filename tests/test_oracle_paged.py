"""Pins of the paged-cache oracle: torch's attention, its complex rotation, plain sorting (CPU)."""

import numpy as np
import torch

from oracle import paged as P

rng = np.random.default_rng(11)


def _cache(lens, page, Hkv, d):
    width = max(-(-n // page) for n in lens)
    n_pages = sum(-(-n // page) for n in lens) + 2
    free = list(rng.permutation(n_pages))
    table = [[free.pop() if i * page < n else -1 for i in range(width)] for n in lens]
    return rng.standard_normal((n_pages, page, Hkv, d)), rng.standard_normal((n_pages, page, Hkv, d)), table


def test_attention_is_torch_attention_of_the_gathered_rows():
    lens, cu, page, Hq, Hkv, d = [37, 16, 5], [0, 4, 20, 21], 16, 6, 2, 8
    K, V, table = _cache(lens, page, Hkv, d)
    q = rng.standard_normal((21, Hq, d))
    got = P.paged_attention(q, K, V, table, lens, cu, heads_scored=Hkv)
    for b, n in enumerate(lens):
        p, r = P.slot_rows(table[b], n, page)
        k, v = (torch.from_numpy(x[p, r]).permute(1, 0, 2).repeat_interleave(Hq // Hkv, 0) for x in (K, V))
        m = cu[b + 1] - cu[b]
        see = torch.arange(n) <= (n - m) + torch.arange(m)[:, None]
        x = torch.from_numpy(q[cu[b]:cu[b + 1]]).permute(1, 0, 2)
        want = torch.nn.functional.scaled_dot_product_attention(x, k, v, attn_mask=see)
        assert np.allclose(got["o"][cu[b]:cu[b + 1]], want.permute(1, 0, 2).numpy(), atol=1e-12)
        s = (x @ k.transpose(1, 2) * d ** -0.5).masked_fill(~see, -np.inf)
        assert np.allclose(got["lse"][cu[b]:cu[b + 1]], s.logsumexp(-1).T.numpy(), atol=1e-12)
        a = s.softmax(-1).sum(1).view(Hkv, Hq // Hkv, n).sum(1)
        assert np.allclose(got["weights"][b, :, :n], a.numpy(), atol=1e-12)


def test_rows_that_see_nothing_and_empty_sequences():
    K, V, table = _cache([2, 0, 3], 16, 1, 4)
    q = rng.standard_normal((4, 1, 4))
    got = P.paged_attention(q, K, V, table, [2, 0, 3], [0, 4, 4, 4], heads_scored=1)
    assert np.array_equal(got["o"][:2], np.zeros((2, 1, 4))) and np.all(np.isneginf(got["lse"][:2]))
    assert np.allclose(got["o"][2, 0], V[table[0][0], 0, 0]) and np.isclose(got["weights"][0].sum(), 2.0)


def test_append_turns_and_places():
    lens, cu, page, d = [20, 3], [0, 5, 8], 16, 8
    K, V, table = _cache(lens, page, 2, d)
    k, v, pos = rng.standard_normal((8, 2, d)), rng.standard_normal((8, 2, d)), np.arange(8) * 7 + 3
    K1, V1 = P.cache_append(k, v, K, V, table, lens, cu, pos)
    z = torch.view_as_complex(torch.stack((torch.from_numpy(k[..., :4]), torch.from_numpy(k[..., 4:])), -1).contiguous())
    ang = torch.outer(torch.from_numpy(pos).double(), 500000.0 ** (-torch.arange(4).double() / 4))
    z = z * torch.polar(torch.ones_like(ang), ang)[:, None]
    want = torch.cat((z.real, z.imag), -1).numpy()
    at = [(0, 15 + i, i) for i in range(5)] + [(1, i, 5 + i) for i in range(3)]
    for b, t, row in at:
        p, r = table[b][t // page], t % page
        assert np.allclose(K1[p, r], want[row]) and np.array_equal(V1[p, r], v[row])
        K1[p, r], V1[p, r] = K[p, r], V[p, r]
    assert np.array_equal(K1, K) and np.array_equal(V1, V)


def test_evict_keeps_what_sorting_keeps():
    lens, page = [40, 7], 16
    K, V, table = _cache(lens, page, 2, 4)
    w = rng.integers(0, 5, (2, 2, 48)).astype(np.float64)  # many ties
    n_pages = K.shape[0]
    K, V = (np.concatenate((x, np.zeros((2, page, 2, 4)))) for x in (K, V))
    dst = [[n_pages], [n_pages + 1]]
    K1, V1, w1, new, kept = P.cache_evict(K, V, table, lens, w, 12, 2, 3, dst, 16)
    assert new == [12, 7] and list(kept[1, 0]) == list(range(7)) + [-1] * 5
    for h in range(2):
        idx = kept[0, h]
        assert list(idx[:2]) == [0, 1] and list(idx[-3:]) == [37, 38, 39] and np.all(np.diff(idx) > 0)
        free, out = w[0, h, 2:37], sorted(set(range(2, 37)) - set(idx))
        assert np.array_equal(np.sort(w[0, h, idx[2:-3]]), np.sort(free)[-7:])
        low = w[0, h, idx[2:-3]].min()
        assert all(w[0, h, j] < low or (w[0, h, j] == low and j > max(i for i in idx[2:-3] if w[0, h, i] == low))
                   for j in out)
        p, r = P.slot_rows(table[0], 40, page)
        assert np.array_equal(K1[n_pages, :12, h], K[p[idx], r[idx], h])
        assert np.array_equal(w1[0, h], np.concatenate((w[0, h, idx], np.zeros(4))))
