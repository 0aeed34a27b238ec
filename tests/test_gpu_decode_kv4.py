"""Sparse decode over a 4-bit cache (GPU) against attention in fp64 over the
values the cache stands for, and the serving-step operators run together."""
import math

import numpy as np
import pytest
import torch

import sparse_attention_aware_b200 as sa
from sparse_attention_aware_b200 import spans as SP
from tests import step_ref as R

pytestmark = pytest.mark.gpu

DEVICE_FAULT = 5


def _cache(seed, B, hkv, d, page, lens, extra=3):
    g = torch.Generator().manual_seed(seed)
    per = max(1, -(-max(lens) // page))
    pages = B * per + extra
    kv = R.random_records(g, pages, hkv, page, d)
    table = torch.randperm(pages, generator=g)[:B * per].view(B, per).int()
    return g, kv, table, torch.tensor(lens, dtype=torch.int32)


def _gpu(kv, table, lens, dev):
    return sa.PagedCache4(kv.to(dev), table.to(dev), lens.to(dev))


def _token_lists(g, B, H, lens, kcap, full=False):
    idx, cnt = np.full((B, H, kcap), -1, dtype=np.int32), np.zeros((B, H), dtype=np.int32)
    for b in range(B):
        for h in range(H):
            n = min(kcap, lens[b])
            if not full:
                n = int(torch.randint(0, n + 1, (1,), generator=g))
            cnt[b, h] = n
            idx[b, h, :n] = torch.randperm(lens[b], generator=g)[:n].sort().values.numpy() if n else []
    return torch.from_numpy(idx), torch.from_numpy(cnt)


TOKEN_CASES = [  # seed, B, Hq, Hkv, d, page, lens, kcap, splits, f32
    (1, 1, 1, 1, 128, 16, [1], 1, 1, False), (2, 1, 4, 4, 64, 16, [300], 256, 0, True),
    (3, 3, 8, 2, 128, 16, [40, 1, 777], 64, 3, False), (4, 2, 12, 3, 128, 64, [1500, 90], 1200, 1, True),
    (5, 4, 5, 1, 64, 64, [0, 17, 2000, 63], 333, 7, False), (6, 1, 2, 2, 128, 16, [5000], 2600, 2, False)]


@pytest.mark.parametrize("seed,B,H,hkv,d,page,lens,kcap,splits,f32", TOKEN_CASES)
def test_token_lists(cuda_dev, seed, B, H, hkv, d, page, lens, kcap, splits, f32):
    g, kv, table, sl = _cache(seed, B, hkv, d, page, lens)
    q = torch.randn(B, H, d, generator=g)
    q = q if f32 else q.bfloat16()
    idx, cnt = _token_lists(g, B, H, lens, kcap, full=seed % 2 == 0)
    scale = 1 / math.sqrt(d)
    ref = R.decode(kv, table, q, lambda b, h: idx[b, h, :cnt[b, h]], scale)
    ws = sa.Workspace(cuda_dev)
    got = sa.sparse_decode_attn(_gpu(kv, table, sl, cuda_dev), q.to(cuda_dev),
                                sa.TokenSelection(idx.to(cuda_dev), cnt.to(cuda_dev)), scale, splits, ws=ws)
    assert ws.status()[0] == 0
    R.check_decode(got, ref)
    empty = (cnt == 0)
    assert bool((got[0].cpu()[empty] == 0).all()) and bool(torch.isinf(got[1].cpu()[empty]).all())


BLOCK_CASES = [  # seed, B, Hq, Hkv, d, page, lens, spans per sequence, splits, f32
    (11, 1, 1, 1, 128, 16, [1], [[(0, 1)]], 1, False),
    (12, 2, 8, 1, 128, 16, [900, 30], [[(0, 900)], [(3, 29)]], 0, False),
    (13, 3, 32, 2, 64, 16, [500, 0, 64], [[(0, 4), (100, 333), (490, 500)], [], [(15, 17)]], 4, True),
    (14, 2, 6, 2, 128, 64, [2000, 129], [[(0, 2000)], [(0, 129)]], 1, True),
    (15, 1, 20, 1, 128, 64, [1111], [[(1, 2), (63, 65), (128, 1100)]], 3, False),
    (16, 2, 40, 1, 64, 64, [700, 65], [[(0, 700)], [(64, 65)]], 2, False),
    (17, 2, 64, 8, 128, 16, [4100, 1500], [[(0, 4), (3076, 4100)], [(988, 1500)]], 0, False),
    (18, 1, 4, 4, 128, 64, [6000], [[(0, 6000)]], 64, False),
    (19, 2, 4, 2, 128, 16, [4100, 3], [[(0, 4100)], [(0, 3)]], 1, False),
    (20, 1, 3, 1, 64, 16, [5555], [[(1, 5554)]], 3, True),
    (26, 1, 16, 1, 128, 64, [9000], [[(0, 9000)]], 2, True)]


@pytest.mark.parametrize("seed,B,H,hkv,d,page,lens,spans,splits,f32", BLOCK_CASES)
def test_block_lists(cuda_dev, seed, B, H, hkv, d, page, lens, spans, splits, f32):
    g, kv, table, sl = _cache(seed, B, hkv, d, page, lens)
    q = torch.randn(B, H, d, generator=g)
    q = q if f32 else q.bfloat16()
    blocks, cnt = R.pack_entries([R.entries_of(s, n, page) for s, n in zip(spans, lens)])
    scale = 0.7 / math.sqrt(d)
    toks = [torch.cat([torch.arange(a, e) for a, e in s]) if s else torch.zeros(0) for s in spans]
    ref = R.decode(kv, table, q, lambda b, h: toks[b], scale)
    ws = sa.Workspace(cuda_dev)
    c = _gpu(kv, table, sl, cuda_dev)
    sel = sa.BlockSelection(blocks.to(cuda_dev), cnt.to(cuda_dev))
    got = sa.sparse_decode_attn(c, q.to(cuda_dev), sel, scale, splits, ws=ws)
    assert ws.status()[0] == 0
    R.check_decode(got, ref)
    again = sa.sparse_decode_attn(c, q.to(cuda_dev), sel, scale, splits, ws=ws)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_scores_far_apart(cuda_dev):
    """Rising and falling scores of thousands: the running maximum moves by far
    more than its slack, and most weights underflow."""
    B, H, d, page, n = 1, 2, 128, 16, 1600
    g, kv, table, sl = _cache(21, B, 1, d, page, [n])
    k = torch.randn(n, d, generator=g).double() * 0.01
    k[:, 0] += torch.linspace(-40, 40, n).double()
    v = torch.randn(n, d, generator=g).double()
    t = torch.arange(n)
    kv[table[0, t // page].long(), 0, t % page] = R.records(k, v)
    q = torch.randn(B, H, d, generator=g)
    q[0, 0, 0], q[0, 1, 0] = 100.0, -100.0
    q = q.bfloat16()
    blocks, cnt = R.pack_entries([R.entries_of([(0, n)], n, page)])
    idx = t.int().expand(B, H, n).contiguous()
    for sel in (sa.BlockSelection(blocks.to(cuda_dev), cnt.to(cuda_dev)),
                sa.TokenSelection(idx.to(cuda_dev), torch.full((B, H), n, dtype=torch.int32, device=cuda_dev))):
        for splits in (1, 5):
            got = sa.sparse_decode_attn(_gpu(kv, table, sl, cuda_dev), q.to(cuda_dev), sel, 1.0, splits)
            R.check_decode(got, R.decode(kv, table, q, lambda b, h: t, 1.0))


@pytest.mark.parametrize("scale,size", [(0.0, 1.0), (-0.15, 1.0), (0.09, 1e-25), (0.09, 0.0), (1e-12, 1e12)])
@pytest.mark.parametrize("f32", [False, True])
def test_scales_and_queries_of_every_size(cuda_dev, scale, size, f32):
    """A scale of zero or below, queries far below and above one, and of zeros."""
    g, kv, table, sl = _cache(29, 2, 2, 64, 16, [90, 333])
    q = torch.randn(2, 6, 64, generator=g) * size
    q[1, 3] = 0
    q = q if f32 else q.bfloat16()
    blocks, cnt = R.pack_entries([R.entries_of([(0, n)], n, 16) for n in (90, 333)])
    idx = torch.arange(90).int().expand(2, 6, 90).contiguous()
    for sel, toks in ((sa.BlockSelection(blocks.to(cuda_dev), cnt.to(cuda_dev)), lambda b, h: torch.arange((90, 333)[b])),
                      (sa.TokenSelection(idx.to(cuda_dev), torch.full((2, 6), 90, dtype=torch.int32, device=cuda_dev)),
                       lambda b, h: torch.arange(90))):
        got = sa.sparse_decode_attn(_gpu(kv, table, sl, cuda_dev), q.to(cuda_dev), sel, scale)
        R.check_decode(got, R.decode(kv, table, q, toks, scale))


def test_a_pool_past_32_bits(cuda_dev):
    """Records, bf16 rows and slots whose byte offsets pass 2^32: append, expand and decode there."""
    d, page, hkv, T = 128, 64, 1, 150
    g = torch.Generator().manual_seed(30)
    pages = 520_000                              # 4.8 GB of records
    high = torch.tensor([519_999, 480_001, 470_003], dtype=torch.int32)
    slots = (high.long()[torch.arange(T) // page] * page + torch.arange(T) % page).to(cuda_dev)
    assert int(slots.min()) * (d + 16) > 2 ** 32
    x = torch.randn(T, 3, d, generator=g).bfloat16()
    table, lens = high[None].to(cuda_dev), torch.tensor([T], dtype=torch.int32, device=cuda_dev)
    pos = torch.arange(T).int()
    inv = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float()
    kv = torch.zeros(pages, hkv, page, d + 16, dtype=torch.uint8, device=cuda_dev)
    c = sa.PagedCache4(kv, table, lens)
    xd = x.to(cuda_dev)
    ws = sa.Workspace(cuda_dev)
    q = sa.rope_append(c, xd[:, :1], xd[:, 1:2], xd[:, 2:], pos.to(cuda_dev), slots, inv.to(cuda_dev), ws=ws)
    rec = R.records(R.norm_rope(x[:, 1:2], None, 0, pos, inv, False), x[:, 2:].double())
    assert torch.equal(kv[table[0].long()].cpu().transpose(1, 2).reshape(-1, hkv, d + 16)[:T], rec)
    assert int(kv[:470_000].count_nonzero()) == 0
    rk, rv, _ = R.values(rec)
    k16, v16 = sa.expand_kv4(c, table[0], ws=ws)
    assert torch.equal(k16.cpu().transpose(1, 2).reshape(-1, hkv, d)[:T], rk.bfloat16())
    small = kv[table[0].long()].cpu()
    blocks, cnt = R.pack_entries([R.entries_of([(0, T)], T, page)])
    ql = q[-1:].contiguous()
    ref = R.decode(small, torch.tensor([[0, 1, 2]]), ql.cpu(), lambda b, h: torch.arange(T), 0.1)
    idx = torch.arange(T).int().view(1, 1, T).to(cuda_dev)
    for sel in (sa.BlockSelection(blocks.to(cuda_dev), cnt.to(cuda_dev)),
                sa.TokenSelection(idx, torch.full((1, 1), T, dtype=torch.int32, device=cuda_dev))):
        R.check_decode(sa.sparse_decode_attn(c, ql, sel, 0.1, ws=ws), ref)
    del kv, c
    kp = torch.zeros(300_000, hkv, page, d, dtype=torch.bfloat16, device=cuda_dev)   # 4.9 GB
    vp = torch.zeros_like(kp)
    top = torch.tensor([299_999, 280_001, 290_003], dtype=torch.int64)
    slots = (top[torch.arange(T) // page] * page + torch.arange(T) % page).to(cuda_dev)
    c = sa.PagedCache(kp, vp, table, lens)
    sa.rope_append(c, xd[:, :1], xd[:, 1:2], xd[:, 2:], pos.to(cuda_dev), slots, ws=ws)
    for pool, row in ((kp, 1), (vp, 2)):
        got = pool[top.to(cuda_dev)].transpose(1, 2).reshape(-1, hkv, d)[:T]
        assert torch.equal(got, xd[:, row:row + 1]) and int(pool[:280_000].count_nonzero()) == 0
    ws.raise_on_fault("past 32 bits")


@pytest.mark.parametrize("splits", [1, 3])
def test_value_scales_far_apart(cuda_dev, splits):
    """Value rows from 2^-40 to 2^20 of one another, rising, falling and mixed, with
    the weight on small ones: each head's error stays within its own rows' share."""
    d, page, n = 128, 16, 700
    for order in ("rising", "falling", "mixed"):
        g, kv, table, sl = _cache(27, 1, 1, d, page, [n])
        e = torch.linspace(-40, 20, n).double()
        e = e if order == "rising" else e.flip(0) if order == "falling" else e[torch.randperm(n, generator=g)]
        v = torch.randn(n, d, generator=g).double() * 2.0 ** e[:, None]
        k = torch.randn(n, d, generator=g).double() * 0.05
        k[:, 0] -= 0.08 * (e + 40) / 60 * 40     # the larger the values, the smaller the weight
        t = torch.arange(n)
        kv[table[0, t // page].long(), 0, t % page] = R.records(k, v)
        q = torch.zeros(1, 2, d)
        q[:, :, 0], q[:, 1, 1] = 10.0, 1.0
        blocks, cnt = R.pack_entries([R.entries_of([(0, n)], n, page)])
        sel = sa.BlockSelection(blocks.to(cuda_dev), cnt.to(cuda_dev))
        out, lse = sa.sparse_decode_attn(_gpu(kv, table, sl, cuda_dev), q.to(cuda_dev), sel, 1.0, splits)
        ref = R.decode(kv, table, q, lambda b, h: t, 1.0)
        # share of row t in the output: its weight times its largest value; each is kept
        # to 2^-11 (2^-8 in all with the bf16 output), or to 2^-31 of the largest scale
        rk, rv, s = R.values(kv[table[0, t // page].long(), 0, t % page])
        for h in range(2):
            w = torch.softmax(rk @ q[0, h].double(), 0)
            share = (w[:, None] * (rv.abs() + 15 * s[:, 1].repeat_interleave(d // 2, 1))).sum(0)
            lim = 2.0 ** -10 * share + R.BF16_HALF * ref[0][0, h].abs() + w.sum() * 2.0 ** -31 * float(s[:, 1].max()) * 15
            err = (out[0, h].double().cpu() - ref[0][0, h]).abs()
            assert bool((err <= lim).all()), (order, h, float((err / lim).max()))


def test_calls_on_two_streams(cuda_dev):
    """Decodes queued on two streams at once, without workspaces, equal the same calls alone."""
    g, kv, table, sl = _cache(28, 3, 2, 128, 16, [3000, 700, 1999])
    c = _gpu(kv, table, sl, cuda_dev)
    blocks, cnt = R.pack_entries([R.entries_of([(0, n)], n, 16) for n in (3000, 700, 1999)])
    sel = sa.BlockSelection(blocks.to(cuda_dev), cnt.to(cuda_dev))
    qs = torch.randn(2, 20, 3, 8, 128, generator=g).bfloat16().to(cuda_dev)
    alone = [[sa.sparse_decode_attn(c, q, sel, num_splits=5) for q in side] for side in qs]
    torch.cuda.synchronize(cuda_dev)
    streams = [torch.cuda.Stream(cuda_dev) for _ in range(2)]
    got = [[], []]
    for i in range(20):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[j].append(sa.sparse_decode_attn(c, qs[j, i], sel, num_splits=5))
    torch.cuda.synchronize(cuda_dev)
    for a, b in zip(alone, got):
        for x, y in zip(a, b):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_unordered_and_repeated_tokens(cuda_dev):
    """A list is a multiset: any order, and a token named twice counts twice."""
    g, kv, table, sl = _cache(22, 1, 1, 64, 16, [100])
    q = torch.randn(1, 1, 64, generator=g)
    idx = torch.tensor([[[99, 3, 3, 50, 0, 3, 98]]], dtype=torch.int32)
    got = sa.sparse_decode_attn(_gpu(kv, table, sl, cuda_dev), q.to(cuda_dev),
                                sa.TokenSelection(idx.to(cuda_dev), torch.tensor([[7]], dtype=torch.int32,
                                                                                 device=cuda_dev)), 0.2, 2)
    R.check_decode(got, R.decode(kv, table, q, lambda b, h: idx[0, 0], 0.2))


def test_bad_device_data_is_skipped_and_recorded(cuda_dev):
    page, d = 16, 128
    g, kv, table, sl = _cache(23, 2, 1, d, page, [80, 80])
    q = torch.randn(2, 2, d, generator=g).bfloat16()
    scale = 0.1
    c = _gpu(kv, table, sl, cuda_dev)
    idx = torch.arange(40).int().expand(2, 2, 40).clone()
    idx[0, 1, 7], idx[1, 0, 39] = 80, -3
    cnt = torch.full((2, 2), 40, dtype=torch.int32)
    keep = lambda b, h: [t for t in idx[b, h].tolist() if 0 <= t < 80]
    ws = sa.Workspace(cuda_dev)
    got = sa.sparse_decode_attn(c, q.to(cuda_dev), sa.TokenSelection(idx.to(cuda_dev), cnt.to(cuda_dev)), scale, 2, ws=ws)
    st, det = ws.status()
    assert st == DEVICE_FAULT and det[1] == 3
    R.check_decode(got, R.decode(kv, table, q, keep, scale))
    # a page out of range, for both kinds of list
    bad = table.clone()
    bad[1, 2] = kv.shape[0]
    c = _gpu(kv, bad, sl, cuda_dev)
    toks = lambda b, h: [t for t in range(40) if not (b == 1 and t // page == 2)]
    blocks, bc = R.pack_entries([R.entries_of([(0, 40)], 80, page)] * 2)
    for sel in (sa.TokenSelection(torch.arange(40).int().expand(2, 2, 40).contiguous().to(cuda_dev), cnt.to(cuda_dev)),
                sa.BlockSelection(blocks.to(cuda_dev), bc.to(cuda_dev))):
        got = sa.sparse_decode_attn(c, q.to(cuda_dev), sel, scale, 1, ws=ws)
        st, det = ws.status()
        assert st == DEVICE_FAULT and det[1] == 2
        R.check_decode(got, R.decode(kv, table, q, toks, scale))
    # malformed entries, an entry past the length, and counts out of range
    c = _gpu(kv, table, sl, cuda_dev)
    blocks, bc = R.pack_entries([R.entries_of([(0, 40)], 80, page), R.entries_of([(0, 40)], 80, page)], 6)
    blocks[0, 1], blocks[1, 0], blocks[1, 2] = torch.tensor([1, 9, 4, 16]), torch.tensor([77, 0, 16, 0]), \
        torch.tensor([4, 0, 17, 32])
    got = sa.sparse_decode_attn(c, q.to(cuda_dev), sa.BlockSelection(blocks.to(cuda_dev), bc.to(cuda_dev)), scale, 3,
                                ws=ws)
    assert ws.status()[1][1] == 5
    skip = {0: (1,), 1: (0, 2)}
    R.check_decode(got, R.decode(kv, table, q, lambda b, h: [t for t in range(40) if t // page not in skip[b]], scale))
    cnt[0, 0], cnt[1, 1] = 41, -1
    got = sa.sparse_decode_attn(c, q.to(cuda_dev), sa.TokenSelection(
        torch.arange(40).int().expand(2, 2, 40).contiguous().to(cuda_dev), cnt.to(cuda_dev)), scale, 1, ws=ws)
    assert ws.status()[1][1] == 4
    R.check_decode(got, R.decode(kv, table, q, lambda b, h: range(0 if (b, h) == (1, 1) else 40), scale))
    sl[0] = 10 ** 6
    got = sa.sparse_decode_attn(_gpu(kv, table, sl, cuda_dev), q.to(cuda_dev), sa.BlockSelection(
        *[x.to(cuda_dev) for x in R.pack_entries([R.entries_of([(0, 40)], 80, page)] * 2)]), scale, 1, ws=ws)
    assert ws.status()[1][1] == 1
    R.check_decode(got, R.decode(kv, table, q, lambda b, h: range(40), scale))


def test_garbage_in_unselected_rows_does_not_reach_the_output(cuda_dev):
    """Rows outside the list may hold anything (their parameters NaN and inf here)."""
    g, kv, table, sl = _cache(24, 1, 2, 128, 64, [200])
    q = torch.randn(1, 4, 128, generator=g).bfloat16()
    blocks, cnt = R.pack_entries([R.entries_of([(5, 70), (130, 131)], 200, 64)])
    toks = list(range(5, 70)) + [130]
    ref = R.decode(kv, table, q, lambda b, h: toks, 0.1)
    dirty = kv.clone()
    mask = torch.ones(kv.shape[0], 64, dtype=torch.bool)
    for t in toks:
        mask[table[0, t // 64].long(), t % 64] = False
    dirty[mask.nonzero()[:, 0], :, mask.nonzero()[:, 1]] = 0xff       # codes 15, parameters NaN
    sel = sa.BlockSelection(blocks.to(cuda_dev), cnt.to(cuda_dev))
    R.check_decode(sa.sparse_decode_attn(_gpu(dirty, table, sl, cuda_dev), q.to(cuda_dev), sel, 0.1, 2), ref)


@pytest.mark.parametrize("splits", [1, 4])
def test_a_row_that_is_not_a_number_shows(cuda_dev, splits):
    """A selected row stored as NaN makes its heads' outputs NaN and no others'."""
    g, kv, table, sl = _cache(25, 2, 2, 128, 16, [64, 64])
    bad = torch.full((1, 128), float("nan")).double()
    kv[table[0, 1].long(), 1, 5] = R.records(bad, torch.randn(1, 128, generator=g).double())[0]
    q = torch.randn(2, 4, 128, generator=g).bfloat16()
    blocks, cnt = R.pack_entries([R.entries_of([(0, 64)], 64, 16)] * 2)
    one = torch.full((2, 4, 1), 21, dtype=torch.int32)
    for sel in (sa.BlockSelection(blocks.to(cuda_dev), cnt.to(cuda_dev)),
                sa.TokenSelection(one.to(cuda_dev), torch.ones(2, 4, dtype=torch.int32, device=cuda_dev))):
        out, lse = sa.sparse_decode_attn(_gpu(kv, table, sl, cuda_dev), q.to(cuda_dev), sel, 0.1, splits)
        assert torch.isnan(out[0, 2:]).all() and torch.isnan(lse[0, 2:]).all()
        assert torch.isfinite(out[0, :2]).all() and torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all()


def test_a_step_of_a_served_batch(cuda_dev):
    """The operators together, as a serving loop runs them: plan, append into a
    4-bit cache, span selection, decode; prompts first, then single tokens, with
    a sequence that ends and one that is admitted; and the pages expanded for
    the bf16 top-k and decode."""
    g = torch.Generator().manual_seed(31)
    B, hq, hkv, d, page, num_pages, cap = 3, 8, 2, 128, 16, 40, 128
    i32 = dict(dtype=torch.int32, device=cuda_dev)
    table, lens = torch.zeros((B, 16), **i32), torch.zeros(B, **i32)
    pool = sa.PagePool.full(num_pages, page, cuda_dev)
    cache = sa.PagedCache4.empty(num_pages, hkv, page, d, table, lens)
    inv = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float()
    w = (1 + 0.1 * torch.randn(2, d, generator=g)).bfloat16()
    ws = sa.Workspace(cuda_dev)
    plan = sa.AppendPlan.empty(B, cap, cuda_dev)
    hist = [[torch.zeros(0, hkv, d).double()] * 2 for _ in range(B)]     # plain: keys, values stored so far
    scale = 1 / math.sqrt(d)
    for new in ([50, 0, 33], [1, 20, 1], [1, 1, 1], [-1, 1, 1], [17, 1, 1], [1, 1, 1]):
        n = sum(max(x, 0) for x in new)
        qkv = torch.randn(n, hq + 2 * hkv, d, generator=g).bfloat16()
        pad = torch.zeros(cap, hq + 2 * hkv, d, dtype=torch.bfloat16)
        pad[:n] = qkv
        x = pad.to(cuda_dev)
        sa.plan_append(table, lens, torch.tensor(new, **i32), pool, cap, plan=plan, ws=ws)
        q = sa.rope_append(cache, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], plan.positions, plan.slots,
                           inv.to(cuda_dev), q_weight=w[0].to(cuda_dev), k_weight=w[1].to(cuda_dev), ws=ws)
        last = (plan.cu_tokens[1:] - 1).clamp(min=0).long()
        ql = q[last]                                                     # each sequence's newest query
        prod = [SP.spans_for(SP.GLOBAL, int(m)) for m in lens.tolist()]
        spans, cnt, rnd = SP.pack(prod, cuda_dev)
        sel = sa.select_blocks_spans(cache, spans, cnt, rnd, ws=ws)
        out, lse = sa.sparse_decode_attn(cache, ql, sel, scale, 0, ws=ws)
        ws.raise_on_fault("step")
        # plain
        at = 0
        for b, m in enumerate(new):
            if m < 0:
                hist[b] = [torch.zeros(0, hkv, d).double()] * 2
                continue
            start = hist[b][0].shape[0]
            pos = torch.arange(start, start + m)
            kk = R.norm_rope(qkv[at:at + m, hq:hq + hkv], w[1], 1e-6, pos, inv, False)
            rec = R.records(kk, qkv[at:at + m, hq + hkv:].double())
            rk, rv, _ = R.values(rec)
            hist[b] = [torch.cat([hist[b][0], rk]), torch.cat([hist[b][1], rv])]
            at += m
        assert lens.tolist() == [len(x[0]) for x in hist]
        assert int(pool.free_count) == num_pages - sum(-(-len(x[0]) // page) for x in hist)
        kv, t, qc = cache.kv.cpu(), table.cpu(), ql.cpu()
        for b in range(B):
            m = len(hist[b][0])
            tok = torch.arange(m)
            rk, rv, _ = R.values(kv[t[b, tok // page].long(), :, tok % page])
            assert torch.equal(rk, hist[b][0]) and torch.equal(rv, hist[b][1])
        R.check_decode((out, lse), R.decode(kv, t, qc, lambda b, h: torch.arange(len(hist[b][0])), scale))
    # the pages as a bf16 cache for the top-k and the bf16 decode
    pages = torch.arange(num_pages, **i32)
    k16, v16 = sa.expand_kv4(cache, pages)
    c16 = sa.PagedCache(k16, v16, table, lens)
    top = sa.select_topk(c16, ql, 16, ws=ws)
    o16, l16 = sa.sparse_decode_attn(c16, ql, top, scale, 1, ws=ws)
    o4, l4 = sa.sparse_decode_attn(cache, ql, top, scale, 1, ws=ws)
    ws.raise_on_fault("bf16 copy")
    idx, cnt = top.idx.cpu(), top.count.cpu()
    R.check_decode((o4, l4), R.decode(kv, t, qc, lambda b, h: idx[b, h, :cnt[b, h]], scale))
    # bf16 pages round each value by half a step: so much may the two differ
    assert float((o16.float() - o4.float()).abs().max()) <= 2.0 ** -5 and float((l16 - l4).abs().max()) <= 2.0 ** -5


def test_a_captured_step_replays(cuda_dev):
    """Plan, append, span selection and decode captured in one graph: each
    replay is the next step of the loop."""
    g = torch.Generator().manual_seed(41)
    B, hq, hkv, d, page, num_pages, steps = 2, 8, 2, 64, 16, 20, 20
    i32 = dict(dtype=torch.int32, device=cuda_dev)
    inv = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float().to(cuda_dev)
    xs = torch.randn(steps, B, hq + 2 * hkv, d, generator=g).bfloat16().to(cuda_dev)

    def setup():
        table, lens = torch.zeros((B, 8), **i32), torch.zeros(B, **i32)
        pool = sa.PagePool.full(num_pages, page, cuda_dev)
        return table, lens, pool, sa.PagedCache4.empty(num_pages, hkv, page, d, table, lens)

    spans = torch.tensor([[[0, 1 << 20]]] * B, **i32)
    one = torch.ones(B, **i32)
    rnd = torch.zeros((B, 1), dtype=torch.uint8, device=cuda_dev)
    ws = sa.Workspace(cuda_dev)

    def step(st, x, plan, blk, out, lse, qo):
        table, lens, pool, cache = st
        sa.plan_append(table, lens, one, pool, B, plan=plan, ws=ws)
        sa.rope_append(cache, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], plan.positions, plan.slots, inv,
                       q_out=qo, ws=ws)
        sa.select_blocks_spans(cache, spans, one, rnd, out=blk, ws=ws)
        sa.sparse_decode_attn(cache, qo, blk, 0.125, 0, out=out, lse=lse, ws=ws)

    def buffers():
        return (sa.AppendPlan.empty(B, B, cuda_dev),
                sa.BlockSelection(torch.empty((B, 16, 4), **i32), torch.empty(B, **i32)),
                torch.empty((B, hq, d), dtype=torch.bfloat16, device=cuda_dev),
                torch.empty((B, hq), dtype=torch.float32, device=cuda_dev),
                torch.empty((B, hq, d), dtype=torch.bfloat16, device=cuda_dev))

    eager = []
    st, bufs = setup(), buffers()
    for i in range(steps):
        step(st, xs[i], *bufs)
        eager.append((bufs[2].clone(), bufs[3].clone()))
    torch.cuda.synchronize(cuda_dev)
    stream = torch.cuda.Stream(cuda_dev)
    st2, bufs2, x = setup(), buffers(), xs[0].clone()
    stream.wait_stream(torch.cuda.current_stream(cuda_dev))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(st2, x, *bufs2)
    for i in range(steps):
        x.copy_(xs[i])
        graph.replay()
        assert torch.equal(bufs2[2], eager[i][0]) and torch.equal(bufs2[3], eager[i][1]), i
    ws.raise_on_fault("graph")
    assert st2[1].tolist() == [steps] * B and torch.equal(st2[3].kv, st[3].kv) and torch.equal(st2[0], st[0])
    del graph


@pytest.mark.parametrize("heads,d,page,f32", [(1, 128, 64, False), (2, 64, 16, True), (3, 128, 16, False), (4, 128, 64, False),
                                              (4, 64, 64, False), (4, 128, 16, True), (5, 128, 64, False), (8, 64, 16, False)])
@pytest.mark.parametrize("only", ["both", "first", "second", "odd"])
def test_neighbouring_tiles_of_16_rows_far_apart(cuda_dev, heads, d, page, f32, only):
    """Every other 16 rows hold keys and values of another size: each head puts its
    weight on the one kind or the other, and lists may hold one kind alone."""
    hkv, n = 2, 64 * 21
    g, kv, table, sl = _cache(31 + heads, 2, hkv, d, page, [n, n - 13])
    t = torch.arange(n)
    second = (t // 16 % 2 == 1)
    for b in range(2):
        for h in range(hkv):
            k, v = torch.randn(2, n, d, generator=g).double()
            k[:, 0] = torch.where(second, -6.0, 6.0).double()
            v[second] *= 8
            kv[table[b, t // page].long(), h, t % page] = R.records(k, v)
    q = torch.randn(2, hkv * heads, d, generator=g)
    q[:, ::2, 0], q[:, 1::2, 0] = 30.0, -30.0
    q = q if f32 else q.bfloat16()
    spans, toks = [], []
    for m in (n, n - 13):
        if only == "both":
            s = [(0, m)]
        elif only == "odd":
            s = [(64 * i + 5, min(64 * i + 5 + 11 * (i % 5), m)) for i in range(21) if 64 * i + 5 < m and i % 5]
        else:
            s = [(i, min(i + 16, m)) for i in range(16 * (only == "second"), m, 32)]
        spans.append(s)
        toks.append(torch.cat([torch.arange(a, e) for a, e in s]))
    blocks, cnt = R.pack_entries([R.entries_of(s, m, page) for s, m in zip(spans, (n, n - 13))])
    c = _gpu(kv, table, sl, cuda_dev)
    ref = R.decode(kv, table, q, lambda b, h: toks[b], 1 / math.sqrt(d))
    for splits in (0, 1, 3):
        ws = sa.Workspace(cuda_dev)
        got = sa.sparse_decode_attn(c, q.to(cuda_dev), sa.BlockSelection(blocks.to(cuda_dev), cnt.to(cuda_dev)),
                                    1 / math.sqrt(d), splits, ws=ws)
        assert ws.status()[0] == 0
        R.check_decode(got, ref, (only, splits))
    H, most = hkv * heads, max(len(x) for x in toks)
    idx = torch.full((2, H, most), -1, dtype=torch.int32)
    for b in range(2):
        idx[b, :, :len(toks[b])] = toks[b].int()
    num = torch.tensor([len(x) for x in toks], dtype=torch.int32)[:, None].expand(2, H).contiguous()
    for splits in (0, 2):
        R.check_decode(sa.sparse_decode_attn(c, q.to(cuda_dev), sa.TokenSelection(idx.to(cuda_dev), num.to(cuda_dev)),
                                             1 / math.sqrt(d), splits), ref, (only, "lists", splits))


@pytest.mark.parametrize("heads", [2, 8])
def test_odd_and_even_channels_far_apart(cuda_dev, heads):
    """Channels at their rows' smallest value beside channels at the largest, odd or
    even ones: each comes out to its own bf16 rounding (all rows' values are alike)."""
    d, page, n = 128, 16, 500
    for low in (0, 1):
        g, kv, table, sl = _cache(41, 1, 1, d, page, [n])
        t = torch.arange(n)
        v = torch.full((n, d), 60.0).double()
        v[:, low::2] = 0.25
        kv[table[0, t // page].long(), 0, t % page] = R.records(torch.randn(n, d, generator=g).double(), v)
        _, rv, _ = R.values(kv[table[0, t // page].long(), 0, t % page])
        q = torch.randn(1, heads, d, generator=g).bfloat16()
        blocks, cnt = R.pack_entries([R.entries_of([(0, n)], n, page)])
        out, _ = sa.sparse_decode_attn(_gpu(kv, table, sl, cuda_dev), q.to(cuda_dev),
                                       sa.BlockSelection(blocks.to(cuda_dev), cnt.to(cuda_dev)), 0.05)
        # all rows alike: the output is the row.  A small channel is z p / p beside sums of
        # codes that cancel exactly (its code is 0); a large one has its weights' 2^-11 and the output's 2^-8
        want = rv[0].expand(1, heads, d)
        lim = want.abs() * (R.BF16_HALF + torch.where(torch.arange(d) % 2 == low, 2.0 ** -18, 2.0 ** -10))
        assert bool(((out.double().cpu() - want).abs() <= lim).all())


def test_graphs_replayed_side_by_side(cuda_dev):
    """Two graphs captured one after the other without workspaces, replayed on two
    streams at once: neither's parts reach the other's output."""
    g, kv, table, sl = _cache(43, 3, 2, 128, 16, [3000, 700, 1999])
    c = _gpu(kv, table, sl, cuda_dev)
    blocks, cnt = R.pack_entries([R.entries_of([(0, n)], n, 16) for n in (3000, 700, 1999)])
    sel = sa.BlockSelection(blocks.to(cuda_dev), cnt.to(cuda_dev))
    qs = torch.randn(2, 3, 8, 128, generator=g).bfloat16().to(cuda_dev)
    alone = [sa.sparse_decode_attn(c, q, sel, num_splits=5) for q in qs]
    torch.cuda.synchronize(cuda_dev)
    side, graphs, got = torch.cuda.Stream(cuda_dev), [], []
    with torch.cuda.stream(side):
        sa.sparse_decode_attn(c, qs[0], sel, num_splits=5)
    torch.cuda.synchronize(cuda_dev)
    for q in qs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            for _ in range(20):
                out = sa.sparse_decode_attn(c, q, sel, num_splits=5)
        got.append(out)
    streams = [torch.cuda.Stream(cuda_dev) for _ in range(2)]
    for _ in range(20):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize(cuda_dev)
        for a, b in zip(alone, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
