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
