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
