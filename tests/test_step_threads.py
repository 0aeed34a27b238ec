"""Two threads' calls on one workspace: while one is between asking for its address
and having launched, the other may outgrow the buffer, whose memory stays (CPU; the
library's functions are stand-ins)."""
import gc
import threading
import time
import weakref

import pytest
import torch

import sparse_attention_aware_b200 as sa
from sparse_attention_aware_b200 import api

I32 = dict(dtype=torch.int32)


class Library:
    """A library each of whose calls runs ``during``."""

    def __init__(self, during):
        self.during = during

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 512

        def call(*a):
            self.during()
            return 0
        return call


def _calls(ws):
    table, lens = torch.zeros((2, 3), **I32), torch.zeros(2, **I32)
    c = sa.PagedCache4.empty(6, 2, 16, 64, table, lens)
    c16 = sa.PagedCache(*(torch.zeros(6, 2, 16, 64).bfloat16() for _ in range(2)), table, lens)
    x = torch.zeros(2, 8, 64).bfloat16()
    pos, slots = torch.zeros(2, **I32), torch.zeros(2, dtype=torch.int64)
    sel = sa.TokenSelection(torch.zeros((2, 4, 3), **I32), torch.zeros((2, 4), **I32))
    q = x[:, :4].contiguous()
    spans = torch.zeros((2, 1, 2), **I32)
    return dict(
        plan=lambda: sa.plan_append(table, lens, lens, sa.PagePool.full(6, 16, "cpu"), 4, ws=ws),
        append=lambda: sa.rope_append(c, x[:, :4], x[:, 4:6], x[:, 6:], pos, slots, ws=ws),
        append16=lambda: sa.rope_append(c16, x[:, :4], x[:, 4:6], x[:, 6:], pos, slots, ws=ws),
        expand=lambda: sa.expand_kv4(c, pos, ws=ws),
        decode4=lambda: sa.sparse_decode_attn(c, q, sel, ws=ws),
        decode=lambda: sa.sparse_decode_attn(c16, q, sel, ws=ws),
        topk=lambda: sa.select_topk(c16, q, 3, ws=ws),
        spans=lambda: sa.select_blocks_spans(c16, spans, lens, torch.zeros((2, 1), dtype=torch.uint8), ws=ws))


@pytest.mark.parametrize("name", ["plan", "append", "append16", "expand", "decode4", "decode", "topk", "spans"])
def test_a_replaced_buffer_outlives_the_call_that_uses_it(monkeypatch, name):
    ws, during = sa.Workspace("cpu"), [lambda: None]
    monkeypatch.setattr(api.L, "load", lambda *a: Library(lambda: during[0]()))
    monkeypatch.setattr(api, "_fast", None)
    monkeypatch.setattr(api, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(api, "_stream", lambda stream=None: None)
    call = _calls(ws)[name]
    call()                                   # the buffer is there
    first, alive = weakref.ref(ws.buf), []

    def outgrown():
        t = threading.Thread(target=lambda: ws.get(1 << 20))
        t.start()
        t.join()
        assert ws.buf.numel() > 1 << 20 and ws.buf is not first()
        alive.append(first() is not None)

    during[0] = outgrown
    call()
    assert alive == [True]
    gc.collect()
    assert first() is None                   # and not longer


def test_threads_that_outgrow_a_buffer_at_once(monkeypatch):
    """Each gets one that is large enough, and all share the last."""
    ws = sa.Workspace("cpu")
    zeros = ws._zeros
    monkeypatch.setattr(ws, "_zeros", lambda n: (time.sleep(0.05), zeros(n))[1])
    got, gate = {}, threading.Barrier(6)

    def one(n):
        gate.wait()
        got[n] = ws.at(n, 0)

    threads = [threading.Thread(target=one, args=(1 << (10 + i),)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(got[n][1] >= n for n in got) and len(got) == 6
    assert ws.at(1 << 15, 0)[0] == got[1 << 15][0]
