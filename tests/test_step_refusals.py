"""The serving-step entry points refuse what they cannot take, on the host and
before any launch (CPU), and their plain 64-bit forms hold their own pins."""
import ctypes
import math

import pytest
import torch

import sparse_attention_aware_b200 as sa
from sparse_attention_aware_b200 import _lib as L
from sparse_attention_aware_b200 import api
from sparse_attention_aware_b200 import build as B
from tests import step_ref as R

OK, INV, UNS, WS = 0, 1, 2, 3
WSP, WSN = 0x100000, 1 << 30     # fake, aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def kv4(batch=2, Hkv=2, d=128, P=16, max_pages=8, num_pages=16, kv=0x10000):
    return L.KV4CacheS(kv, 0x20000, 0x30000, batch, Hkv, d, P, max_pages, num_pages)


def kv16(batch=2, Hkv=2, d=128, P=16, max_pages=8, num_pages=16):
    return L.KVCacheS(0x10000, 0x18000, 0x20000, 0x30000, batch, Hkv, d, P, max_pages, num_pages)


def plan_args(**kw):
    f = dict(page_table=0x1000, seq_lens=0x2000, new_lens=0x3000, free_pages=0x4000, free_count=0x5000,
             seq_lens_out=0x6000, free_count_out=0x7000, cu_tokens=0x8000, positions=0x9000, slots=0xa000,
             seq_ids=0xb000, batch=3, page_size=16, max_pages_per_seq=8, num_pages=24, num_free=24, max_tokens=10)
    f.update(kw)
    return L.PlanArgsS(**f)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), INV), (dict(num_free=-1), INV), (dict(max_tokens=-1), INV), (dict(num_pages=-1), INV),
    (dict(page_size=32), UNS), (dict(batch=4097), UNS), (dict(max_pages_per_seq=1 << 27), UNS),
    (dict(free_count=None), INV), (dict(free_count_out=None), INV), (dict(cu_tokens=None), INV),
    (dict(page_table=None), INV), (dict(seq_lens=None), INV), (dict(new_lens=None), INV),
    (dict(seq_lens_out=None), INV), (dict(positions=None), INV), (dict(slots=None), INV),
    (dict(slots=0xa004), INV), (dict(positions=0x9002), INV), (dict(free_pages=None), INV)])
def test_plan_refusals(lib, kw, want):
    a = plan_args(**kw)
    assert lib.sa_plan_append(ctypes.byref(a), WSP, WSN, None) == want


def test_plan_workspace(lib):
    a = plan_args()
    assert lib.sa_plan_append(ctypes.byref(a), None, WSN, None) == WS
    assert lib.sa_plan_append(ctypes.byref(a), WSP, 255, None) == WS
    assert lib.sa_plan_append(ctypes.byref(a), WSP + 16, WSN, None) == WS
    assert lib.sa_plan_append(None, WSP, WSN, None) == INV


def append_args(**kw):
    f = dict(q=0x40000, k=0x50000, v=0x60000, q_stride=1024, k_stride=256, v_stride=256, q_out=0x70000,
             q_out_stride=1024, positions=0x80000, slots=0x90000, inv_freq=0xa0000, q_weight=0xb0000,
             k_weight=0xc0000, weight_dtype=L.DTYPE_BF16, eps=1e-6, num_tokens=4, num_q_heads=8, rot_dim=128,
             interleaved=0)
    f.update(kw)
    return L.AppendArgsS(**f)


@pytest.mark.parametrize("kw,want", [
    (dict(num_tokens=-1), INV), (dict(num_q_heads=0), INV), (dict(rot_dim=24), INV), (dict(rot_dim=144), INV),
    (dict(rot_dim=-16), INV), (dict(weight_dtype=7), INV), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV),
    (dict(eps=math.inf), INV), (dict(inv_freq=None), INV), (dict(q=None), INV), (dict(k=None), INV),
    (dict(v=None), INV), (dict(q_out=None), INV), (dict(positions=None), INV), (dict(slots=None), INV),
    (dict(q_stride=1020), INV), (dict(k_stride=252), INV), (dict(v_stride=1), INV), (dict(q_out_stride=1016), INV),
    (dict(q=0x40008), INV), (dict(q_out=0x70002), INV), (dict(q_weight=0xb0008), INV), (dict(slots=0x90004), INV),
    (dict(q_out=0x40000, q_stride=2048), INV)])
@pytest.mark.parametrize("four", [False, True])
def test_append_refusals(lib, kw, want, four):
    a = append_args(**kw)
    c = kv4() if four else kv16()
    fn = lib.sa_rope_append_kv4 if four else lib.sa_rope_append
    assert fn(ctypes.byref(c), ctypes.byref(a), WSP, WSN, None) == want


def test_append_cache_and_workspace(lib):
    a = append_args()
    for c, fn in ((kv4(d=96), lib.sa_rope_append_kv4), (kv4(P=32), lib.sa_rope_append_kv4),
                  (kv16(d=96), lib.sa_rope_append), (kv16(P=8), lib.sa_rope_append),
                  (kv4(Hkv=64, num_pages=1 << 24, P=64), lib.sa_rope_append_kv4)):
        assert fn(ctypes.byref(c), ctypes.byref(a), WSP, WSN, None) == UNS
    assert lib.sa_rope_append_kv4(ctypes.byref(kv4(kv=0x10008)), ctypes.byref(a), WSP, WSN, None) == INV
    assert lib.sa_rope_append_kv4(ctypes.byref(kv4(kv=None)), ctypes.byref(a), WSP, WSN, None) == INV
    assert lib.sa_rope_append_kv4(ctypes.byref(kv4()), ctypes.byref(a), WSP, 0, None) == WS
    assert lib.sa_rope_append(ctypes.byref(kv16()), None, WSP, WSN, None) == INV
    # a call without tokens launches nothing
    z = append_args(num_tokens=0)
    assert lib.sa_rope_append(ctypes.byref(kv16()), ctypes.byref(z), WSP, WSN, None) == OK
    assert lib.sa_rope_append_kv4(ctypes.byref(kv4()), ctypes.byref(z), WSP, WSN, None) == OK


def test_expand_refusals(lib):
    f = lambda c=None, pages=0x1000, n=3, k=0x2000, v=0x3000, ws=WSP, wn=WSN: lib.sa_expand_kv4(
        ctypes.byref(c or kv4()), pages, n, k, v, ws, wn, None)
    assert f(n=-1) == INV and f(pages=None) == INV and f(k=None) == INV and f(v=None) == INV
    assert f(k=0x2008) == INV and f(pages=0x1002) == INV and f(c=kv4(kv=0x10004, batch=0)) == INV
    assert f(c=kv4(d=80)) == UNS and f(ws=None) == WS and f(wn=128) == WS
    assert f(n=0, pages=None, k=None, v=None) == OK


def test_decode_refusals(lib):
    def f(c=None, q=0x40000, dt=L.DTYPE_BF16, Hq=8, sel=None, scale=0.1, splits=1, out=0x50000, lse=None, ws=WSP,
          wn=WSN):
        sel = sel or L.SelectionS(L.SEL_TOKENS, 0x60000, 0x70000, 16, None, None, 0)
        return lib.sa_sparse_decode_attn_kv4(ctypes.byref(c or kv4()), q, dt, Hq, ctypes.byref(sel), scale, splits, out,
                                             lse, ws, wn, None)
    assert f(c=kv4(d=96)) == UNS and f(c=kv4(P=32)) == UNS and f(Hq=3) == UNS
    assert f(c=kv4(Hkv=64, num_pages=1 << 24, P=64), Hq=64) == UNS
    assert f(c=kv4(batch=70000)) == UNS
    assert f(splits=-1) == INV and f(splits=65) == INV and f(q=None) == INV and f(q=0x40004) == INV
    assert f(out=None) == INV and f(dt=5) == INV and f(scale=math.nan) == INV and f(scale=math.inf) == INV
    assert f(lse=0x50002) == INV and f(c=kv4(kv=None)) == INV and f(c=kv4(kv=0x10008)) == INV
    assert f(sel=L.SelectionS(9, 0x60000, 0x70000, 16, None, None, 0)) == INV
    assert f(sel=L.SelectionS(L.SEL_TOKENS, None, 0x70000, 16, None, None, 0)) == INV
    assert f(sel=L.SelectionS(L.SEL_BLOCKS, None, None, 0, 0x60008, 0x70000, 4)) == INV
    assert f(sel=L.SelectionS(L.SEL_BLOCKS, None, None, 0, 0x60000, None, 4)) == INV
    assert f(ws=None) == WS and f(wn=256) == WS and f(splits=0, wn=256) == WS


def test_decode_workspace_covers_the_chosen_splits(lib):
    for batch, Hkv, Hq in ((1, 1, 1), (1, 8, 64), (4, 8, 64), (32, 8, 32), (700, 4, 32), (1, 2, 40)):
        c = kv4(batch=batch, Hkv=Hkv)
        auto = lib.sa_kv4_decode_workspace_bytes(ctypes.byref(c), Hq, 0)
        assert auto % 256 == 0 and auto >= lib.sa_kv4_decode_workspace_bytes(ctypes.byref(c), Hq, 1) > 256
        assert auto <= lib.sa_kv4_decode_workspace_bytes(ctypes.byref(c), Hq, 64)
    bad = kv4()
    assert lib.sa_kv4_decode_workspace_bytes(ctypes.byref(bad), 3, 0) == 0
    assert lib.sa_kv4_decode_workspace_bytes(ctypes.byref(bad), 8, 65) == 0
    assert lib.sa_kv4_decode_workspace_bytes(ctypes.byref(kv4(d=32)), 8, 1) == 0


def test_spans_take_a_cache_without_pools(lib):
    """The span selection reads lengths and page geometry alone; the other modes still need the pools."""
    c = kv16()
    c.k = c.v = None
    a = L.BlockSelectArgsS()
    a.mode = L.SEL_SPANS
    q = L.WsQueryS(0, 0, 0, 0, ctypes.pointer(a))
    assert lib.sa_workspace_bytes(L.OP_SELECT_BLOCKS, ctypes.byref(c), ctypes.byref(q)) == 256
    a.mode = L.SEL_RBS
    assert lib.sa_workspace_bytes(L.OP_SELECT_BLOCKS, ctypes.byref(c), ctypes.byref(q)) == 0
    o = L.BlockListS()
    assert lib.sa_select_blocks(ctypes.byref(c), ctypes.byref(a), ctypes.byref(o), WSP, WSN, None) == INV
    a.mode, a.max_spans = L.SEL_SPANS, 2000
    assert lib.sa_select_blocks(ctypes.byref(c), ctypes.byref(a), ctypes.byref(o), WSP, WSN, None) == INV


# ---------------------------------------------------------------------------
# the binding's own checks
# ---------------------------------------------------------------------------
def _cache4(d=128, pages=6, B=2):
    return sa.PagedCache4.empty(pages, 2, 16, d, torch.zeros(B, 3, dtype=torch.int32),
                                torch.zeros(B, dtype=torch.int32))


def test_cache4_checks():
    c = _cache4()
    assert (c.batch, c.num_kv_heads, c.page_size, c.head_dim, c.max_pages, c.num_pages) == (2, 2, 16, 128, 3, 6)
    s = api.kv4_struct(c)
    assert (s.head_dim, s.num_pages, s.page_size) == (128, 6, 16)
    with pytest.raises(ValueError):
        api.kv4_struct(sa.PagedCache4(c.kv.to(torch.int8), c.page_table, c.seq_lens))
    with pytest.raises(ValueError):
        api.kv4_struct(sa.PagedCache4(c.kv[..., :100], c.page_table, c.seq_lens))
    with pytest.raises(ValueError):
        api.kv4_struct(sa.PagedCache4(c.kv, c.page_table.long(), c.seq_lens))
    with pytest.raises(ValueError):
        api.kv4_struct(sa.PagedCache4(c.kv, c.page_table, c.seq_lens[:1]))
    with pytest.raises(ValueError):
        api.kv4_struct(c, torch.device("cuda:0"))


def test_binding_refusals():
    c = _cache4()
    q = torch.zeros(5, 4, 128, dtype=torch.bfloat16)
    k = torch.zeros(5, 2, 128, dtype=torch.bfloat16)
    pos, slot = torch.zeros(5, dtype=torch.int32), torch.zeros(5, dtype=torch.int64)
    bad = [dict(q=q.float()), dict(k=k[:4]), dict(v=k[..., :64]), dict(positions=pos.long()),
           dict(slots=slot.int()), dict(inv_freq=torch.zeros(64, dtype=torch.float64)),
           dict(q_weight=torch.ones(64)), dict(q_weight=torch.ones(128, dtype=torch.float64)),
           dict(q_weight=torch.ones(128), k_weight=torch.ones(128, dtype=torch.bfloat16)),
           dict(q_out=torch.zeros(5, 4, 128)), dict(q_out=torch.zeros(5, 128, 4, dtype=torch.bfloat16).mT)]
    for kw in bad:
        args = dict(cache=c, q=q, k=k, v=k, positions=pos, slots=slot)
        args.update(kw)
        with pytest.raises((ValueError, TypeError)):
            sa.rope_append(**args)
    with pytest.raises(ValueError):      # a view that cannot be updated in place
        w = torch.zeros(5, 8, 128, dtype=torch.bfloat16)[:, ::2]
        sa.rope_append(c, w, k, k, pos, slot, q_out=w)
    with pytest.raises(ValueError):      # another head_dim than the cache's
        sa.rope_append(_cache4(64), q, k, k, pos, slot)
    sel = sa.TokenSelection(torch.zeros(2, 4, 8, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        sa.sparse_decode_attn(c, q[:2, :, :64].contiguous(), sel)
    with pytest.raises(ValueError):
        sa.sparse_decode_attn(c, q[:3], sel)
    with pytest.raises(ValueError):
        sa.sparse_decode_attn(c, q[:2, :2], sel)
    with pytest.raises(ValueError):
        sa.expand_kv4(c, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        sa.expand_kv4(c, torch.zeros(2, dtype=torch.int32), k=torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16))
    pool = sa.PagePool.full(6, 16, "cpu")
    assert pool.free_pages.tolist() == [5, 4, 3, 2, 1, 0] and int(pool.free_count) == 6
    with pytest.raises(ValueError):
        sa.plan_append(c.page_table, c.seq_lens, torch.zeros(3, dtype=torch.int32), pool, 4)
    with pytest.raises(ValueError):
        sa.plan_append(c.page_table, c.seq_lens, c.seq_lens, pool, 4,
                       plan=sa.AppendPlan.empty(2, 5, "cpu"))
    with pytest.raises(sa.SAError):      # top-k reads bf16 pages
        sa.workspace_bytes(L.OP_SELECT_TOPK, c, num_q_heads=4, k=8)
    with pytest.raises(TypeError, match="expand_kv4"):
        sa.select_topk(c, q[:2], 4)
    with pytest.raises(TypeError, match="expand_kv4"):
        sa.select_blocks_rbs(c, q)


def test_rows_layouts():
    packed = torch.zeros(6, 9, 64, dtype=torch.bfloat16)
    dev = packed.device
    for x, st, same in ((packed[:, 2:6], 9 * 64, True), (packed[::2, :4], 2 * 9 * 64, True),
                        (packed[:, ::2], 5 * 64, False), (packed[:1, :3], 3 * 64, True),
                        (packed[:1, :4].expand(6, 4, 64), 0, True),
                        (packed[..., 1:].new_zeros(6, 4, 65)[..., 1:], 4 * 64, False)):
        y, got = api._rows(x, "q", tuple(x.shape), dev)
        assert got == st and (y is x) == same


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def test_plain_record_pins():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(50, 128, generator=g).double()
    k, v, s = R.values(R.records(x, 3 * x + 1))
    for got, ref, i in ((k, x, 0), (v, 3 * x + 1, 1)):
        step = s[:, i].repeat_interleave(64, dim=1)
        # half a step of the code, and the zero's own rounding (2^-8 of the minimum); the top code clamps
        lim = step * (0.5 + 15 * 2.0 ** -8) + 2.0 ** -8 * ref.abs().amax(1, keepdim=True)
        assert bool(((got - ref).abs() <= lim).all())
    # a constant row, and one of 16 equal steps, come back as they are
    assert torch.equal(R.values(R.records(torch.full((1, 64), -3.5).double(), x[:1, :64]))[0],
                       torch.full((1, 64), -3.5).double())
    ramp = (torch.arange(64) % 16).double()[None] * 0.25 - 2
    assert torch.equal(R.values(R.records(ramp, ramp))[1], ramp)
    # ties go to the even code: 0.5, 1.5, 2.5 steps
    t = torch.tensor([0.0, 0.5, 1.5, 2.5, 15.0] + [0.0] * 59).double()[None]
    c, p = R.quantize(torch.cat([t[:, :32], t[:, :32]], 1))
    assert c[0, :5].tolist() == [0, 0, 2, 2, 15] and float(p[0, 0, 0]) == 1.0
    bad = t.clone()
    bad[0, 3] = math.inf
    assert torch.isnan(R.values(R.records(bad, t))[0][0, :32]).all()
    assert torch.isfinite(R.values(R.records(bad, t))[0][0, 32:]).all()


def test_plain_rope_pins():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(4, 3, 64, generator=g).bfloat16()
    inv = 10000.0 ** (-torch.arange(0, 32, 2).float() / 32)
    for il in (False, True):
        z = R.norm_rope(x, None, 0, torch.zeros(4), inv, il)
        assert torch.equal(z, x.double())                       # position 0 turns nothing
        y = R.norm_rope(x, None, 0, torch.arange(4) * 1000, inv, il)
        assert torch.allclose(y.norm(dim=-1), x.double().norm(dim=-1))
        assert torch.equal(y[..., 32:], x.double()[..., 32:])
    # q . k depends on the distance of their positions alone
    a = R.norm_rope(x, None, 0, torch.full((4,), 17), inv, False)
    b = R.norm_rope(x.flip(0), None, 0, torch.full((4,), 5), inv, False)
    a2 = R.norm_rope(x, None, 0, torch.full((4,), 1017), inv, False)
    b2 = R.norm_rope(x.flip(0), None, 0, torch.full((4,), 1005), inv, False)
    assert torch.allclose((a * b).sum(-1), (a2 * b2).sum(-1), atol=1e-9)


def test_plain_plan_pins():
    table = torch.full((3, 4), -1, dtype=torch.int32)
    table[0, :2] = torch.tensor([7, 3])
    table[2, :1] = 5
    free = torch.tensor([9, 8, 1, 0, -1, -1, -1, -1], dtype=torch.int32)
    (t, lens, f, n), (cu, pos, slots, seq) = R.plan(table, torch.tensor([20, 0, 16]), torch.tensor([-1, 18, 1]),
                                                    free, 4, 16, 21)
    # the ended sequence's pages 7, 3 go onto the stack and come off it first
    assert t.tolist()[1][:2] == [3, 7] and t.tolist()[2][:2] == [5, 0] and n == 3
    assert lens.tolist() == [0, 18, 17] and cu.tolist() == [0, 0, 18, 19]
    assert slots[0] == 48 and slots[17] == 7 * 16 + 1 and slots[18] == 0 and slots[19] == -1
    assert pos[17] == 17 and pos[18] == 16 and seq[18] == 2 and seq[20] == -1
