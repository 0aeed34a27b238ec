"""The serving-step calls captured into graphs: the memory whose addresses a graph
holds, and what its replays record (GPU)."""
import pytest
import torch

import sparse_attention_aware_b200 as sa
from sparse_attention_aware_b200 import api
from tests import step_ref as R

pytestmark = pytest.mark.gpu

DEVICE_FAULT, CAPACITY = 5, 7


def _plan_inputs(dev, B=3):
    i32 = dict(dtype=torch.int32, device=dev)
    return dict(page_table=torch.zeros((B, 4), **i32), seq_lens=torch.zeros(B, **i32),
                new_lens=torch.ones(B, **i32), pool=sa.PagePool.full(12, 16, dev), max_tokens=4)


def _grow(ws, dev, nbytes=1 << 20):
    """A later eager call that outgrows the workspace."""
    raw = torch.cuda.current_stream(dev).cuda_stream
    before = ws.buf.data_ptr()
    api._scratch(ws, dev, None, nbytes)
    assert ws.buf.data_ptr() != before and raw in ws._raw


def test_an_outgrown_workspace_still_takes_the_records_of_replays(cuda_dev):
    s = _plan_inputs(cuda_dev)
    ws = sa.Workspace(cuda_dev)
    sa.plan_append(**s, ws=ws)                      # the short way from here on
    stream = torch.cuda.Stream(cuda_dev)
    stream.wait_stream(torch.cuda.current_stream(cuda_dev))
    with torch.cuda.stream(stream):
        sa.plan_append(**s, ws=ws)
    torch.cuda.synchronize(cuda_dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        sa.plan_append(**s, ws=ws)
    held = ws.buf.data_ptr()
    _grow(ws, cuda_dev)
    assert [b.data_ptr() for b in ws._kept] == [held]
    s["new_lens"].fill_(2)                          # 6 tokens, 4 fit
    lens = s["seq_lens"].tolist()
    graph.replay()
    assert ws.status() == (CAPACITY, (CAPACITY, 13, 6)) and s["seq_lens"].tolist() == lens
    assert ws.status()[0] == 0
    s["new_lens"].fill_(1)
    graph.replay()
    assert ws.status()[0] == 0 and s["seq_lens"].tolist() == [n + 1 for n in lens]
    del graph


def test_captured_calls_go_the_long_way(cuda_dev, monkeypatch):
    """...which marks the workspace as one that a graph holds."""
    taken = []

    class Spy:
        def __getattr__(self, name):
            def call(*a):
                got = getattr(real, name)(*a)
                taken.append((name, got is not None))
                return got
            return call

    real = api._load_fast()
    assert real is not None
    monkeypatch.setattr(api, "_fast", Spy())
    i32 = dict(dtype=torch.int32, device=cuda_dev)
    g = torch.Generator().manual_seed(1)
    kv = R.random_records(g, 6, 2, 16, 64).to(cuda_dev)
    c = sa.PagedCache4(kv, torch.arange(6, **i32).view(2, 3), torch.tensor([40, 20], **i32))
    x = torch.randn(2, 8, 64, generator=g).bfloat16().to(cuda_dev)
    blocks, cnt = R.pack_entries([R.entries_of([(0, n)], n, 16) for n in (40, 20)])
    sel = sa.BlockSelection(blocks.to(cuda_dev), cnt.to(cuda_dev))
    pages, pos = torch.arange(3, **i32), torch.tensor([39, 19], **i32)
    slots = torch.tensor([5, -1], device=cuda_dev)
    s = _plan_inputs(cuda_dev)
    ws = sa.Workspace(cuda_dev)
    stream = torch.cuda.Stream(cuda_dev)

    def step():
        sa.plan_append(**s, ws=ws)
        q = sa.rope_append(c, x[:, :4], x[:, 4:6], x[:, 6:], pos, slots, ws=ws)
        return sa.expand_kv4(c, pages, ws=ws) + sa.sparse_decode_attn(c, q, sel, ws=ws)

    with torch.cuda.stream(stream):
        step()
        taken.clear()
        ref = step()
    assert {n for n, took in taken if took} == {"plan", "append", "expand", "decode"} and not ws._in_graph
    torch.cuda.synchronize(cuda_dev)
    taken.clear()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = step()
    assert len(taken) == 4 and not any(took for _, took in taken) and ws._in_graph
    graph.replay()
    torch.cuda.synchronize(cuda_dev)
    assert all(torch.equal(a, b) for a, b in zip(ref, got)) and ws.status()[0] == 0
    del graph


def test_first_calls_of_a_captured_stream_record_readably(cuda_dev):
    """Calls without a workspace, the first of their stream, captured: the status is
    clear before any replay, holds the first record until it is read, and is not
    cleared by replays."""
    i32 = dict(dtype=torch.int32, device=cuda_dev)
    g = torch.Generator().manual_seed(2)
    kv = R.random_records(g, 6, 2, 16, 64).to(cuda_dev)
    c = sa.PagedCache4(kv, torch.arange(6, **i32).view(2, 3), torch.tensor([40, 20], **i32))
    q = torch.randn(2, 4, 64, generator=g).bfloat16().to(cuda_dev)
    blocks, cnt = R.pack_entries([R.entries_of([(0, n)], n, 16) for n in (40, 20)])
    sel = sa.BlockSelection(blocks.to(cuda_dev), cnt.to(cuda_dev))
    ref = sa.sparse_decode_attn(c, q, sel, num_splits=2)
    pages, x = torch.arange(3, **i32), torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=cuda_dev)
    slots = torch.tensor([5, -1], device=cuda_dev)
    s = _plan_inputs(cuda_dev)
    used = {k[1] for k in api._default_ws}
    for _ in range(64):                              # a stream that the library has not seen
        stream = torch.cuda.Stream(cuda_dev)
        if stream.cuda_stream not in used:
            break
    torch.cuda.synchronize(cuda_dev)
    sa.device_status(cuda_dev)
    # memory that a buffer of the capture may well get is not zero beforehand
    junk = [torch.full((n,), 0x55, dtype=torch.uint8, device=cuda_dev) for n in (512, 768, 1024, 4096) * 4]
    torch.cuda.synchronize(cuda_dev)
    del junk
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        sa.plan_append(**s)
        sa.rope_append(c, x[:, :4], x[:, 4:6], x[:, 6:], torch.zeros(2, **i32), slots)
        sa.expand_kv4(c, pages)
        out = sa.sparse_decode_attn(c, q, sel, num_splits=2)
    assert sa.device_status(cuda_dev) == (0, (0, 0, 0))
    kv.copy_(R.random_records(torch.Generator().manual_seed(2), 6, 2, 16, 64))
    slots.fill_(-1)
    graph.replay()
    assert sa.device_status(cuda_dev)[0] == 0 and torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    # each call's own fault, recorded by a replay and there after the next
    for bad, chk, value in ((lambda v: slots.fill_(v), 12, 96), (lambda v: pages.fill_(v), 2, 6),
                            (lambda v: sel.blocks[:, 0, 0].fill_(v), 5, 3)):
        good = slots.clone(), pages.clone(), sel.blocks.clone()
        bad(value)
        graph.replay()
        torch.cuda.synchronize(cuda_dev)
        slots.copy_(good[0]), pages.copy_(good[1]), sel.blocks.copy_(good[2])
        s["new_lens"].zero_()
        graph.replay()
        st, det = sa.device_status(cuda_dev)
        assert st == DEVICE_FAULT and det[1] == chk and (chk == 5 or det[2] == value)
        assert sa.device_status(cuda_dev)[0] == 0
    assert torch.equal(out[0], ref[0])
    s["new_lens"].fill_(9)
    graph.replay()
    assert sa.device_status(cuda_dev) == (CAPACITY, (CAPACITY, 13, 27))
    del graph


def test_a_default_workspace_grown_by_a_captured_call(cuda_dev):
    """An older entry point that needs scratch, captured without a workspace after a
    call that needs none: both buffers stay, both records are read."""
    i32 = dict(dtype=torch.int32, device=cuda_dev)
    s = _plan_inputs(cuda_dev)
    c16 = sa.PagedCache(*(torch.randn(6, 2, 16, 64, device=cuda_dev).bfloat16() for _ in range(2)),
                        torch.arange(6, **i32).view(2, 3), torch.tensor([40, 20], **i32))
    q = torch.randn(2, 4, 64, device=cuda_dev)
    spans = torch.tensor([[[0, 40]], [[0, 20]]], **i32)
    sel = sa.select_blocks_spans(c16, spans, torch.ones(2, **i32), torch.zeros((2, 1), dtype=torch.uint8, device=cuda_dev))
    ref = sa.sparse_decode_attn(c16, q, sel, num_splits=8)
    used = {k[1] for k in api._default_ws}
    for _ in range(64):
        stream = torch.cuda.Stream(cuda_dev)
        if stream.cuda_stream not in used:
            break
    torch.cuda.synchronize(cuda_dev)
    sa.device_status(cuda_dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        sa.plan_append(**s)
        out = sa.sparse_decode_attn(c16, q, sel, num_splits=8)
    graph.replay()
    assert sa.device_status(cuda_dev)[0] == 0 and torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    s["new_lens"].fill_(9)
    graph.replay()
    assert sa.device_status(cuda_dev) == (CAPACITY, (CAPACITY, 13, 27))
    s["new_lens"].zero_()
    sel.blocks[:, 0, 0] = 3
    graph.replay()
    st, det = sa.device_status(cuda_dev)
    assert st == DEVICE_FAULT and det[1] == 5
    del graph


def test_a_default_workspace_outgrown_after_the_capture(cuda_dev):
    """Captured without a workspace, then a call on that stream that needs more: a
    replay's record reaches no other tensor, and is read."""
    s = _plan_inputs(cuda_dev)
    i32 = dict(dtype=torch.int32, device=cuda_dev)
    g = torch.Generator().manual_seed(3)
    c = sa.PagedCache4(R.random_records(g, 6, 2, 16, 64).to(cuda_dev), torch.arange(6, **i32).view(2, 3),
                       torch.tensor([40, 20], **i32))
    q = torch.randn(2, 16, 64, generator=g).bfloat16().to(cuda_dev)
    blocks, cnt = R.pack_entries([R.entries_of([(0, n)], n, 16) for n in (40, 20)])
    sel = sa.BlockSelection(blocks.to(cuda_dev), cnt.to(cuda_dev))
    stream = torch.cuda.Stream(cuda_dev)
    stream.wait_stream(torch.cuda.current_stream(cuda_dev))
    with torch.cuda.stream(stream):
        sa.plan_append(**s)
    torch.cuda.synchronize(cuda_dev)
    sa.device_status(cuda_dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        sa.plan_append(**s)
    ws = api._default_ws_at[(cuda_dev.index, stream.cuda_stream)]
    held = ws.buf.data_ptr()
    with torch.cuda.stream(stream):
        while ws.buf.data_ptr() == held:         # (it may have served larger calls before)
            _grow(ws, cuda_dev, 2 * ws.buf.numel())
        sa.sparse_decode_attn(c, q, sel, num_splits=64)
        others = [torch.zeros(n, dtype=torch.uint8, device=cuda_dev) for n in (512, 768, 1024) * 8]
    torch.cuda.synchronize(cuda_dev)
    s["new_lens"].fill_(9)
    graph.replay()
    assert sa.device_status(cuda_dev) == (CAPACITY, (CAPACITY, 13, 27))
    assert not any(bool(x.any()) for x in others)
    del graph
