"""CPU: what the binding takes and hands on, without a GPU."""
import enum
import types

import numpy as np
import pytest
import torch

import selective_state_space_amd as mb


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import os
    if not os.path.exists(mb.lib_path()):
        from selective_state_space_amd import _build
        _build.build()


@pytest.mark.parametrize("kind", [np.int64, np.uint8, np.float64, float, enum.IntEnum("Op", {"x": mb.MB_OP_SSD_CHUNKED})], ids=str)
def test_workspace_size_takes_what_int_takes_as_operator(kind):
    want = mb.mb_workspace_size(mb.MB_OP_SSD_CHUNKED, 2, 100, 4, 64, 1, 64)
    got = mb.mb_workspace_size(kind(mb.MB_OP_SSD_CHUNKED), 2, 100, 4, 64, 1, 64)
    assert want > 0 and type(got) is int and got == want


def test_stream_without_torchs_private_call(monkeypatch):
    """A torch that lacks it: the public call gives the same handle."""
    device = torch.device("cuda", 1)
    seen = []

    def current_stream(d):
        seen.append(d)
        return types.SimpleNamespace(cuda_stream=1234)

    public = types.SimpleNamespace(_C=types.SimpleNamespace(), cuda=types.SimpleNamespace(current_stream=current_stream))
    monkeypatch.setattr(mb, "_torch", lambda: public)
    assert mb._stream(device) == 1234 and seen == [device]
    private = types.SimpleNamespace(_C=types.SimpleNamespace(_cuda_getCurrentRawStream=lambda i: 100 + i))
    monkeypatch.setattr(mb, "_torch", lambda: private)
    assert mb._stream(device) == 101


def test_workspace_of_packed_sequences_holds_their_table():
    """From 65 sequences on (that a workgroup does not find in one look) the sizes allow for a table of segments, 32 bytes
    each beside 8 a sequence; not where every sequence is one segment that its number finds."""
    size = lambda n, T: mb.mb_workspace_size(mb.MB_OP_LINEAR_ATTN, n, T, 512, 64, 512, 64)
    # 512 heads: two workgroups a compute unit are there without cutting a sequence, so there are no states
    assert size(64, 4001) == 0
    assert size(65, 4001) >= 65 * 40 and size(1000, 4001) >= 1000 * 40
    assert size(1000, 1001) == 0 and size(100_000, 1001) == 0
