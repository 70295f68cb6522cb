"""The paged key/value cache's C entry points and binding refuse what they cannot run, before any launch (CPU)."""

import ctypes

# Placeholder addresses: never dereferenced, each case fails an argument
# check on the host before any launch.  A16 is 16-byte aligned, M8 is not.
A16, B16, C16, D16, E16 = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000
M8 = 0x600008


def _paged_cases(S):
    lib, ref = S.lib, ctypes.byref

    def attn(**kw):
        f = dict(dtype=S.BF16, Hq=32, Hkv=8, d=128, scale=0.0)
        f.update(kw)
        return S._lib.AttnDesc(*f.values())

    def cache(**kw):
        f = dict(k_pages=A16, v_pages=B16, num_pages=100, page_stride=0, page_size=16, B=4, page_table=C16, max_pages=8,
                 table_stride=0, seq_lens=D16)
        f.update(kw)
        return S._lib.PagedCache(*f.values())

    def append(a=None, c=None, k=A16, ks=0, v=B16, vs=0, cu=C16, T=5, pos=D16, theta=5e5, ws=None):
        return lambda: lib.spts_cache_append(ref(a or attn()), ref(c or cache()), k, ks, v, vs, cu, T, pos, theta, ws,
                                             None)

    def attend(a=None, c=None, q=A16, qs=0, cu=C16, T=5, o=B16, os=0, lse=None, w=None, Hs=0, wst=0, ws=None, n=0):
        return lambda: lib.spts_paged_attention(ref(a or attn()), ref(c or cache()), q, qs, cu, T, o, os, lse, w, Hs, wst,
                                                ws, n, None)

    def evict(a=None, c=None, w=A16, Hs=8, wst=128, keep=20, sink=1, recent=2, dst=E16, dmax=2, dst_s=0, wo=B16, wos=128,
              nl=D16, kept=None, ws=None, n=0):
        return lambda: lib.spts_cache_evict(ref(a or attn()), ref(c or cache()), w, Hs, wst, keep, sink, recent, dst,
                                            dmax, dst_s, wo, wos, nl, kept, ws, n, None)

    W = 0x800000  # 256-byte aligned
    cases = [
        ("F32 cache", append(a=attn(dtype=S.F32)), S.ERR_UNSUPPORTED, "bf16"),
        ("dtype", append(a=attn(dtype=7)), S.ERR_INVALID, "dtype"),
        ("head dim", attend(a=attn(d=96)), S.ERR_SHAPE, "head dim"),
        ("Hq % Hkv", attend(a=attn(Hq=30)), S.ERR_SHAPE, "Hq"),
        ("group too wide", attend(a=attn(Hq=258, Hkv=2)), S.ERR_UNSUPPORTED, "128"),
        ("NULL pages", evict(c=cache(v_pages=None)), S.ERR_INVALID, "NULL"),
        ("NULL lengths", evict(c=cache(seq_lens=None)), S.ERR_INVALID, "NULL"),
        ("misaligned pages", append(c=cache(k_pages=M8)), S.ERR_INVALID, "misaligned"),
        ("page size 24", attend(c=cache(page_size=24)), S.ERR_UNSUPPORTED, "page_size"),
        ("page size 8", attend(c=cache(page_size=8)), S.ERR_UNSUPPORTED, "page_size"),
        ("page size 512", attend(c=cache(page_size=512)), S.ERR_UNSUPPORTED, "page_size"),
        ("no sequence", attend(c=cache(B=0)), S.ERR_SHAPE, "B"),
        ("too many sequences", attend(c=cache(B=1025)), S.ERR_SHAPE, "B"),
        ("no pages", attend(c=cache(num_pages=0)), S.ERR_SHAPE, "num_pages"),
        ("no table columns", attend(c=cache(max_pages=0)), S.ERR_SHAPE, "max_pages"),
        ("too many slots", attend(c=cache(max_pages=(1 << 26) + 1)), S.ERR_SHAPE, "2^30"),
        ("page stride below a page", append(c=cache(page_stride=16 * 8 * 128 - 8)), S.ERR_SHAPE, "page_stride"),
        ("page stride % 8", append(c=cache(page_stride=16 * 8 * 128 + 4)), S.ERR_SHAPE, "page_stride"),
        ("table stride", append(c=cache(table_stride=7)), S.ERR_SHAPE, "table_stride"),
        ("append T < 0", append(T=-1), S.ERR_SHAPE, "T"),
        ("append NULL rows", append(v=None), S.ERR_INVALID, "NULL"),
        ("append NULL offsets", append(cu=None), S.ERR_INVALID, "NULL"),
        ("append misaligned", append(k=M8), S.ERR_INVALID, "misaligned"),
        ("append k_stride", append(ks=1000), S.ERR_SHAPE, "k_stride"),
        ("append v_stride % 8", append(vs=1030), S.ERR_SHAPE, "v_stride"),
        ("append theta", append(theta=0.0), S.ERR_INVALID, "theta"),
        ("append theta NaN", append(theta=float("nan")), S.ERR_INVALID, "theta"),
        ("append workspace", append(ws=M8), S.ERR_WORKSPACE, "aligned"),
        ("attend T < 0", attend(T=-1), S.ERR_SHAPE, "T"),
        ("attend NULL o", attend(o=None), S.ERR_INVALID, "NULL"),
        ("attend o is q", attend(o=A16), S.ERR_INVALID, "alias"),
        ("attend q_stride", attend(qs=4088), S.ERR_SHAPE, "q_stride"),
        ("attend o_stride % 8", attend(os=4100), S.ERR_SHAPE, "o_stride"),
        ("attend Hs", attend(w=E16, Hs=2, wst=128), S.ERR_SHAPE, "Hs"),
        ("attend w_stride", attend(w=E16, Hs=1, wst=127), S.ERR_SHAPE, "w_stride"),
        ("attend no workspace", attend(), S.ERR_WORKSPACE, "NULL"),
        ("attend workspace too small", attend(ws=W, n=255), S.ERR_WORKSPACE, "needs"),
        ("evict keep 0", evict(keep=0, sink=0, recent=0), S.ERR_SHAPE, "keep"),
        ("evict sink < 0", evict(sink=-1), S.ERR_SHAPE, "sink"),
        ("evict recent < 0", evict(recent=-1), S.ERR_SHAPE, "recent"),
        ("evict sink + recent", evict(sink=10, recent=11), S.ERR_SHAPE, "recent"),
        ("evict Hs", evict(Hs=4), S.ERR_SHAPE, "Hs"),
        ("evict w_stride", evict(wst=100), S.ERR_SHAPE, "w_stride"),
        ("evict w_out_stride", evict(wos=19), S.ERR_SHAPE, "w_out_stride"),
        ("evict weights in place, other stride", evict(wo=A16, wos=256), S.ERR_SHAPE, "strides"),
        ("evict NULL table", evict(dst=None), S.ERR_INVALID, "NULL"),
        ("evict table width", evict(dmax=0), S.ERR_SHAPE, "dst_max_pages"),
        ("evict table stride", evict(dst_s=1), S.ERR_SHAPE, "dst_stride"),
        ("evict same table, other stride", evict(dst=C16, dmax=8, dst_s=9), S.ERR_SHAPE, "strides"),
        ("evict no workspace", evict(), S.ERR_WORKSPACE, "NULL"),
        ("evict workspace too small", evict(ws=W, n=300), S.ERR_WORKSPACE, "needs"),
    ]
    return cases


def test_paged_cache_refusals_return_the_documented_codes():
    import token_skipping_sparse_b200 as S
    before = S.launch_count()
    for name, call, status, text in _paged_cases(S):
        got = call()
        assert got == status, f"{name}: status {got}, want {status} ({S.last_error()})"
        assert text in S.last_error(), f"{name}: message {S.last_error()!r}"
    assert S.launch_count() == before


def test_paged_cache_calls_want_cuda_tensors_of_the_right_kind():
    import pytest
    import torch
    import token_skipping_sparse_b200 as S
    k = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        S.spts_paged_attention(k[0], k, k, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                               torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="page_table"):
        S._lib._paged(k, k, torch.zeros(1, 1), torch.zeros(1, dtype=torch.int32), k.device)
    with pytest.raises(ValueError, match="alike"):
        S._lib._paged(k, k[..., :32], torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), k.device)
    with pytest.raises(ValueError, match="per sequence"):
        S._lib._paged(k, k, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), k.device)


def test_paged_cache_calls_refuse_overlapping_rows():
    """A stride of 0 (a tensor that was expanded) would read as "contiguous" behind the C interface."""
    import pytest
    import torch
    import token_skipping_sparse_b200 as S
    k, table, lens = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(3, 4, dtype=torch.int32), \
        torch.zeros(3, dtype=torch.int32)
    cpu = k.device
    assert S._lib._paged(k, k, table, lens, cpu)[1:] == (2, 64, 3, 16, 4)
    assert S._lib._paged(k[1:].expand(1, 16, 2, 64), k[:1], table[:, 1:], lens, cpu)[5] == 3
    one = k[:1].expand(2, 16, 2, 64)
    with pytest.raises(ValueError, match="pages must not overlap"):
        S._lib._paged(one, one, table, lens, cpu)
    shared = table[:1].expand(3, 4)
    with pytest.raises(ValueError, match="per sequence"):
        S._lib._paged(k, k, shared, lens, cpu)
    with pytest.raises(ValueError, match="per sequence"):
        S._lib._paged(k, k, table, lens[:1].expand(3), cpu)
    with pytest.raises(ValueError, match="overlap"):
        S._lib._table_stride(shared, "dst_table")
    assert S._lib._table_stride(table[:, :2], "dst_table") == 4

    class Here:
        index = cpu.index if cpu.index is not None else -1
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    assert S._lib._packed(q, Here, "q") == 256
    assert S._lib._packed(torch.zeros(5, 6, 64, dtype=torch.bfloat16)[:, 1:5], Here, "q") == 384
    for bad in (q[:1].expand(5, 4, 64), q[:, :1].expand(5, 4, 64), q.transpose(0, 1)):
        with pytest.raises(ValueError, match="overlap"):
            S._lib._packed(bad, Here, "q")
