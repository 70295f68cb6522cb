"""The binding of the paged key/value cache, as far as it runs without a GPU."""

import threading
import time

import pytest
import torch

import token_skipping_sparse_b200 as S

CPU = torch.device("cpu")


@pytest.fixture
def eager(monkeypatch):
    """No graph is captured, and no workspace is cached yet."""
    monkeypatch.setattr(S._lib, "_capturing", lambda: False)
    monkeypatch.setattr(S._lib, "_stream_ws", {})
    return monkeypatch


def test_calls_on_two_streams_have_workspaces_of_their_own(eager):
    a, b = (S._lib._own_ws(None, 1000, CPU, stream) for stream in (7, 8))
    assert a.numel() >= 1000 and b.numel() >= 1000 and a.data_ptr() != b.data_ptr()
    assert not a.any() and not b.any()  # the status words
    # kept as long as they are large enough, replaced by a larger one
    assert S._lib._own_ws(None, 900, CPU, 7) is a
    c = S._lib._own_ws(None, 1001, CPU, 7)
    assert c.numel() >= 1001 and S._lib._own_ws(None, 256, CPU, 7) is c
    assert S._lib._own_ws(None, 256, CPU, 8) is b


def test_a_workspace_that_is_given_is_used(eager):
    ws = torch.zeros(512, dtype=torch.uint8)
    assert S._lib._own_ws(ws, 256, CPU, 7) is ws
    assert not S._lib._stream_ws


class Calls:
    """In the library's place: sizes from it, launches written down."""

    def __init__(self):
        self.seen = []

    def __getattr__(self, name):
        real = getattr(S.lib, name)
        if name.endswith("_workspace"):
            return real

        def call(*args):
            self.seen.append((name,) + args)
            return S.OK
        return call


@pytest.fixture
def host(eager):
    """Calls with tensors on the host, as far as the library."""
    calls = Calls()
    eager.setattr(S._lib, "lib", calls)
    eager.setattr(S._lib, "_elsewhere", lambda dev, who: False)
    eager.setattr(S._lib, "_raw_stream", lambda index: 7)
    eager.setattr(S._lib, "_vector", lambda t, n, dev, what: t.data_ptr())
    return calls


def test_weights_out_has_room_for_the_budget(host):
    k = torch.zeros(600, 16, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 512, dtype=torch.int32), torch.tensor([1000], dtype=torch.int32)
    w = torch.zeros(1, 2, 8192)
    for keep, width, columns in ((2048, 63, 2048), (1008, 63, 1008), (500, 63, 1008), (9000, 63, 8192)):
        _, out = S._lib.spts_cache_evict(k, k.clone(), table, lens, w, keep,
                                         dst_table=torch.zeros(1, width, dtype=torch.int32))
        assert out.shape == (1, 2, columns), (keep, width)


def test_the_first_columns_of_one_sequences_own_table_are_that_table():
    # one row has no stride: nothing but the workspace is missing here
    a = S._lib.AttnDesc(S.BF16, 4, 2, 64, 0.0)

    def status(B, dst_stride):
        c = S._lib.PagedCache(0x100000, 0x200000, 100, 0, 16, B, 0x300000, 8, 0, 0x400000)
        return S.lib.spts_cache_evict(S._lib.C.byref(a), S._lib.C.byref(c), 0x500000, 2, 128, 20, 0, 0, 0x300000, 4,
                                      dst_stride, 0x600000, 128, 0x700000, None, None, 0, None)
    assert status(1, 4) == S.ERR_WORKSPACE and status(1, 8) == S.ERR_WORKSPACE
    assert status(2, 4) == S.ERR_SHAPE and status(2, 8) == S.ERR_WORKSPACE


def test_a_workspace_with_fewer_bytes_than_entries_is_refused(eager):
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(4096), torch.zeros(4096, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            S._lib._own_ws(bad, 256, CPU, 7)


@pytest.mark.parametrize("own", [False, True])
def test_kernels_of_two_threads_do_not_mix_in_one_workspace(host, own):
    # a call that is given no workspace launches all its kernels before another one does
    inside, most = [], []

    def launch(*args):
        inside.append(args[-2])
        most.append(len(inside))
        time.sleep(0.02)
        inside.pop()
        return S.OK
    for name in ("spts_cache_append", "spts_paged_attention", "spts_cache_evict"):
        setattr(host, name, launch)
    k = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16)
    table, lens, cu = torch.arange(8, dtype=torch.int32)[None], torch.tensor([40], dtype=torch.int32), \
        torch.tensor([0, 3], dtype=torch.int32)
    rows, w = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 128)

    def calls():
        ws = torch.zeros(1 << 22, dtype=torch.uint8) if own else None
        for _ in range(3):
            S._lib.spts_cache_append(rows, rows, k, k.clone(), table, lens, cu, ws=ws)
            S._lib.spts_paged_attention(rows, k, k.clone(), table, lens, cu, weights=w, ws=ws)
            S._lib.spts_cache_evict(k, k.clone(), table, lens, w, 20, ws=ws)
    threads = [threading.Thread(target=calls) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(most) == 27 and (max(most) > 1) == own
