"""Workspaces of the serving-step calls: what a captured graph holds the address
of stays (CPU)."""
import weakref

import pytest

import sparse_attention_aware_b200 as sa
from sparse_attention_aware_b200 import api


@pytest.mark.parametrize("again", [False, True])
def test_a_captured_workspace_outgrown_is_kept(monkeypatch, again):
    """A graph holds the address of the workspace that its calls were given.  When a
    later call outgrows it, that memory must not go to another tensor: a replay
    writes its record there."""
    ws = sa.Workspace("cpu")
    if again:                      # the workspace has served its stream before the capture
        ws.at(256, 7)
    monkeypatch.setattr(api, "_capturing", lambda: True, raising=False)
    at = ws.at(256, 7)
    monkeypatch.setattr(api, "_capturing", lambda: False, raising=False)
    first = weakref.ref(ws.buf)
    ws.at(1 << 16, 7)
    assert first() is not None and ws.buf is not first()
    assert any(api._aligned(b) == at[0] for b in ws._kept)
    # an eager buffer that is outgrown is released as before
    second = weakref.ref(ws.buf)
    ws.at(1 << 18, 7)
    assert second() is None and len(ws._kept) == 1
