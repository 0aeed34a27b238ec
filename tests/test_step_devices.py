"""Serving-step calls with a workspace or a stream of another device than their
tensors are refused before a kernel could reach that memory (CPU)."""
import types

import pytest
import torch

import sparse_attention_aware_b200 as sa
from sparse_attention_aware_b200 import api


@pytest.fixture
def handle(monkeypatch):
    """Both devices' current stream is the default one, whose handle is 0."""
    monkeypatch.setattr(api, "_raw_stream", lambda index: 0)
    return 0


def _of(index, nbytes=4096):
    """A workspace whose buffer (never touched) is on that device and has served stream 0."""
    ws = sa.Workspace()
    ws.buf = types.SimpleNamespace(device=torch.device("cuda", index), numel=lambda: nbytes, data_ptr=lambda: 0x10000)
    ws._index, ws._raw = index, {0: (0x10000, nbytes)}
    return ws


def test_another_devices_workspace_is_refused(handle, monkeypatch):
    monkeypatch.setattr(api, "_fast", object())
    here = torch.device("cuda", 0)
    assert api._short(_of(0), here, None)[1:3] == (0x10000, 4096)
    assert api._short(_of(1), here, None) is None
    assert api._scratch(_of(0), here, None, 256)[:3] == (0x10000, 4096, 0)
    for ws in (_of(1), sa.Workspace("cuda:1"), sa.Workspace("cpu")):
        with pytest.raises(ValueError, match="workspace is on"):
            api._scratch(ws, here, None, 256)
    cpu = sa.Workspace("cpu")
    cpu.at(256, 0)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        api._scratch(cpu, here, None, 256)


def test_another_devices_stream_is_refused():
    stream = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        api._scratch(_of(0), torch.device("cuda", 0), stream, 256)
