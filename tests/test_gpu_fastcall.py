"""The binding's native short way (csrc/fastcall.cpp) and its Python way: the
same results, errors and refusals (GPU)."""
import pytest
import torch

import sparse_attention_aware_b200 as sa
from sparse_attention_aware_b200 import api
from tests import step_ref as R

pytestmark = pytest.mark.gpu


class _Spy:
    """The native module, counting the calls that it took."""

    def __init__(self, real):
        self.real, self.taken, self.left = real, [], []

    def __getattr__(self, name):
        def call(*a):
            got = getattr(self.real, name)(*a)
            (self.left if got is None else self.taken).append(name)
            return got
        return call


@pytest.fixture
def spy(monkeypatch):
    real = api._load_fast()
    assert real is not None, "the native calls have not been built"
    s = _Spy(real)
    monkeypatch.setattr(api, "_fast", s)
    return s


def _setup(dev, seed=3):
    g = torch.Generator().manual_seed(seed)
    B, hq, hkv, d, page = 3, 8, 2, 128, 16
    kv = R.random_records(g, 14, hkv, page, d).to(dev)
    table = torch.randperm(14, generator=g)[:12].view(3, 4).int().to(dev)
    lens = torch.tensor([60, 1, 33], dtype=torch.int32, device=dev)
    cache = sa.PagedCache4(kv, table, lens)
    x = torch.randn(B, hq + 2 * hkv, d, generator=g).bfloat16().to(dev)
    inv = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float().to(dev)
    w = (1 + 0.1 * torch.randn(2, d, generator=g)).bfloat16().to(dev)
    idx = torch.zeros(B, hq, 5, dtype=torch.int32)
    idx[0] = torch.randint(0, 60, (hq, 5), generator=g)
    cnt = torch.tensor([[5] * hq, [1] * hq, [0] * hq], dtype=torch.int32)
    blocks, bc = R.pack_entries([R.entries_of([(0, n)], n, page) for n in lens.tolist()])
    return dict(cache=cache, q=x[:, :hq], k=x[:, hq:hq + hkv], v=x[:, hq + hkv:], inv=inv, w=w,
                pos=lens - 1, slots=torch.tensor([5, -1, 200], device=dev),
                tok=sa.TokenSelection(idx.to(dev), cnt.to(dev)), blk=sa.BlockSelection(blocks.to(dev), bc.to(dev)))


def _run(s, ws):
    c = sa.PagedCache4(s["cache"].kv.clone(), s["cache"].page_table.clone(), s["cache"].seq_lens.clone())
    k16, v16 = sa.expand_kv4(c, torch.arange(14, dtype=torch.int32, device=c.kv.device), ws=ws)
    c16 = sa.PagedCache(k16, v16, c.page_table, c.seq_lens)
    pool = sa.PagePool(torch.tensor([13, 12], dtype=torch.int32, device=c.kv.device),
                       torch.tensor([2], dtype=torch.int32, device=c.kv.device), 14, 16)
    p = sa.plan_append(c.page_table, c.seq_lens, torch.tensor([1, -1, 2], dtype=torch.int32, device=c.kv.device), pool,
                       6, ws=ws)
    out = [k16.clone(), v16.clone(), p.cu_tokens, p.positions, p.slots, p.seq_ids, c.page_table, c.seq_lens,
           pool.free_pages, pool.free_count]
    for cc in (c, c16):
        for w in (s["w"], s["w"].float(), None):
            out.append(sa.rope_append(cc, s["q"], s["k"], s["v"], s["pos"], s["slots"], s["inv"],
                                      q_weight=None if w is None else w[0], k_weight=None if w is None else w[1],
                                      eps=1e-5, interleaved=w is None, ws=ws))
    out.append(sa.rope_append(c, s["q"], s["k"], s["v"], s["pos"], s["slots"], ws=ws))
    q = out[-1]
    for sel in (s["tok"], s["blk"]):
        for x in (q, q.float()):
            for kw in ({}, {"num_splits": 0}, {"num_splits": 3, "scale": 0.3}):
                out += sa.sparse_decode_attn(s["cache"], x, sel, ws=ws, **kw)
    o, none = sa.sparse_decode_attn(s["cache"], q, s["blk"], want_lse=False, ws=ws)
    assert none is None
    return out + [o, c.kv, k16, v16]


def test_both_ways_agree(cuda_dev, monkeypatch, spy):
    s = _setup(cuda_dev)
    ws = sa.Workspace(cuda_dev)
    _run(s, ws)                                  # makes the workspace and grows it
    spy.taken.clear(), spy.left.clear()
    a = _run(s, ws)
    assert not spy.left and set(spy.taken) == {"plan", "append", "expand", "decode"}
    monkeypatch.setattr(api, "_fast", None)
    b = _run(s, ws)
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and x.shape == y.shape and torch.equal(x.nan_to_num(), y.nan_to_num())


def test_default_workspaces_are_of_their_stream(cuda_dev, spy):
    """Without a workspace the short way begins with a stream's second call, and
    streams do not share scratch."""
    s = _setup(cuda_dev, 4)
    q = s["q"].contiguous()
    ref = sa.sparse_decode_attn(s["cache"], q, s["blk"], num_splits=2)
    side = torch.cuda.Stream(cuda_dev)
    side.wait_stream(torch.cuda.current_stream(cuda_dev))
    with torch.cuda.stream(side):
        for _ in range(3):
            out = sa.sparse_decode_attn(s["cache"], q, s["blk"], num_splits=2)
    torch.cuda.synchronize(cuda_dev)
    assert torch.equal(ref[0], out[0]) and spy.taken.count("decode") >= 2
    raws = {k[1] for k in api._default_ws_at}
    assert side.cuda_stream in raws and len({id(w) for w in api._default_ws_at.values()}) == len(api._default_ws_at)


def test_the_short_way_leaves_other_calls(cuda_dev, spy):
    """Layouts, types and sizes that the short way does not take get the long
    way's copies or refusals."""
    s = _setup(cuda_dev, 5)
    ws = sa.Workspace(cuda_dev)
    c = s["cache"]
    args = dict(cache=c, q=s["q"], k=s["k"], v=s["v"], positions=s["pos"], slots=s["slots"], inv_freq=s["inv"], ws=ws)
    ref = sa.rope_append(**args)
    spy.taken.clear()
    wide = torch.zeros(3, 16, 128, dtype=torch.bfloat16, device=cuda_dev)
    wide[:, ::2] = s["q"]
    assert torch.equal(sa.rope_append(**{**args, "q": wide[:, ::2]}), ref) and not spy.taken
    for bad in (dict(q=s["q"].float()), dict(positions=s["pos"].long()), dict(slots=s["slots"].int()),
                dict(k=s["k"][:2]), dict(inv_freq=s["inv"].double()), dict(q_weight=s["w"][0][:64]),
                dict(q_weight=s["w"][0].cpu()), dict(q_weight=s["w"][0], k_weight=s["w"][1].float()),
                dict(positions=s["pos"].cpu())):
        with pytest.raises((TypeError, ValueError)):
            sa.rope_append(**{**args, **bad})
    with pytest.raises(sa.SAError):              # rot_dim 8: the library's own refusal, through either way
        sa.rope_append(**{**args, "inv_freq": s["inv"][:4].contiguous()})
    with pytest.raises(sa.SAError):
        sa.rope_append(**{**args, "eps": -1.0})
    q = ref
    for bad in (dict(q=q[:2]), dict(q=q.half()), dict(sel=sa.TokenSelection(s["tok"].idx[:, :4], s["tok"].count)),
                dict(sel=sa.BlockSelection(s["blk"].blocks.long(), s["blk"].block_counts))):
        with pytest.raises((TypeError, ValueError)):
            sa.sparse_decode_attn(**{**dict(cache=c, q=q, sel=s["tok"], ws=ws), **bad})
    for bad in (dict(num_splits=65), dict(num_splits=-1), dict(scale=float("nan"))):
        with pytest.raises(sa.SAError):
            sa.sparse_decode_attn(c, q, s["tok"], ws=ws, **bad)
    with pytest.raises(ValueError):
        sa.expand_kv4(c, torch.zeros(2, dtype=torch.int64, device=cuda_dev), ws=ws)
    with pytest.raises(ValueError):
        sa.plan_append(c.page_table, c.seq_lens, torch.zeros(2, dtype=torch.int32, device=cuda_dev),
                       sa.PagePool.full(4, 16, cuda_dev), 3, ws=ws)
    with pytest.raises((ValueError, RuntimeError)):
        sa.plan_append(c.page_table, c.seq_lens, c.seq_lens, sa.PagePool.full(4, 16, cuda_dev), -3, ws=ws)
    # strided queries are copied
    out = sa.sparse_decode_attn(c, wide[:, ::2], s["blk"], ws=ws)
    assert torch.equal(out[0], sa.sparse_decode_attn(c, s["q"].contiguous(), s["blk"], ws=ws)[0])
