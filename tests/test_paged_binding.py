"""The binding of the paged key/value cache, as far as it runs without a GPU."""

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
