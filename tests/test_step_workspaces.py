"""Workspaces of the serving-step calls -- what a captured graph holds the address
of stays -- and sizes that are refused (CPU)."""
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


def test_sizes_that_ctypes_would_cut_are_refused():
    import torch
    table, lens = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for kw in (dict(num_pages=2 ** 32 + 8), dict(page_size=2 ** 32 + 16), dict(max_tokens=2 ** 31)):
        a = dict(dict(num_pages=8, page_size=16, max_tokens=4), **kw)
        pool = sa.PagePool(torch.arange(8, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), a["num_pages"],
                           a["page_size"])
        with pytest.raises(ValueError, match="32 bits"):
            sa.plan_append(table, lens, lens, pool, a["max_tokens"], ws=sa.Workspace("cpu"))
