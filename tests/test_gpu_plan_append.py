"""Page planning and the norm + rotary append on the GPU against their plain
64-bit forms."""
import pytest
import torch

import sparse_attention_aware_b200 as sa
from tests import step_ref as R

pytestmark = pytest.mark.gpu

DEVICE_FAULT, CAPACITY = 5, 7


# ---------------------------------------------------------------------------
# planning
# ---------------------------------------------------------------------------
def _problem(seed, B, page, most, mix=True):
    """Lengths, new tokens, a shuffled table and a stack that just holds what is needed."""
    g = torch.Generator().manual_seed(seed)
    old = torch.randint(0, most + 1, (B,), generator=g)
    new = torch.randint(0, 2 * page + 3, (B,), generator=g)
    if mix:
        u = torch.rand(B, generator=g)
        new[u < 0.5], new[u < 0.3], new[u < 0.15] = 1, 0, -1
        old[u > 0.9] = 0
    held = (old + page - 1) // page
    per = int(((old + new.clamp(min=0) + page - 1) // page).max()) + 1
    need = int((((old + new + page - 1) // page - held) * (new >= 0)).sum())
    back = int((held * (new < 0)).sum())
    count = max(0, need - back)
    total = int(held.sum()) + count
    perm = torch.randperm(total, generator=g).int()
    table = torch.full((B, per), -77, dtype=torch.int32)
    at = 0
    for b, h in enumerate(held.tolist()):
        table[b, :h] = perm[at:at + h]
        at += h
    free = torch.full((max(total, 1),), -55, dtype=torch.int32)
    free[:count] = perm[at:]
    return table, old.int(), new.int(), free, count, total


@pytest.mark.parametrize("seed,B,page,most", [(1, 1, 16, 0), (2, 1, 64, 700), (3, 7, 16, 100), (4, 33, 16, 3000),
                                              (5, 257, 64, 500), (6, 1030, 16, 90), (7, 4096, 16, 40)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_matches_plain(cuda_dev, seed, B, page, most, in_place):
    table, old, new, free, count, total = _problem(seed, B, page, most)
    tokens = int(new.clamp(min=0).sum())
    cap = tokens + (seed * 7) % 40
    (t, lens, f, n), ref = R.plan(table, old, new, free, count, page, cap)
    ws = sa.Workspace(cuda_dev)
    dt, dl, df = table.to(cuda_dev), old.to(cuda_dev), free.to(cuda_dev)
    pool = sa.PagePool(df, torch.tensor([count], dtype=torch.int32, device=cuda_dev), total, page)
    kw = {}
    if not in_place:
        kw = dict(seq_lens_out=torch.full_like(dl, -9), free_count_out=torch.full_like(pool.free_count, -9))
    p = sa.plan_append(dt, dl, new.to(cuda_dev), pool, cap, ws=ws, **kw)
    assert ws.status()[0] == 0
    got_l = dl if in_place else kw["seq_lens_out"]
    got_n = pool.free_count if in_place else kw["free_count_out"]
    assert torch.equal(dt.cpu(), t) and torch.equal(got_l.cpu(), lens) and int(got_n) == n
    assert torch.equal(df.cpu()[:n], f[:n])
    for x, y in zip((p.cu_tokens, p.positions, p.slots, p.seq_ids), ref):
        assert torch.equal(x.cpu(), y)
    if not in_place:
        assert torch.equal(dl.cpu(), old) and int(pool.free_count) == count


def test_plan_of_long_prompts(cuda_dev):
    """More tokens than one CTA, or eight, take: the same as the plain form."""
    for seed, B, page, most, cap in ((21, 300, 64, 2000, 40001), (22, 9, 16, 9000, 131072), (23, 70, 16, 900, 8000)):
        g = torch.Generator().manual_seed(seed)
        table, old, _, free, _, _ = _problem(seed, B, page, most)
        new = torch.randint(0, 2 * (cap // B), (B,), generator=g)
        new[::7] = -1
        new[new.clamp(min=0).cumsum(0) > cap] = 0
        new = new.int()
        held = (old + page - 1) // page
        per = int(((old + new.clamp(min=0) + page - 1) // page).max()) + 1
        total = int(held.sum()) + cap // page + B + 5
        perm = torch.randperm(total, generator=g).int()
        table, at = torch.full((B, per), -77, dtype=torch.int32), 0
        for b, h in enumerate(held.tolist()):
            table[b, :h] = perm[at:at + h]
            at += h
        free = torch.full((total,), -55, dtype=torch.int32)
        free[:total - at] = perm[at:]
        (t, lens, f, n), ref = R.plan(table, old, new, free, total - at, page, cap)
        ws = sa.Workspace(cuda_dev)
        dt, dl, df = table.to(cuda_dev), old.to(cuda_dev), free.to(cuda_dev)
        pool = sa.PagePool(df, torch.tensor([total - at], dtype=torch.int32, device=cuda_dev), total, page)
        for _ in range(2):                       # and again through the binding's short way, undone in between
            p = sa.plan_append(dt, dl, new.to(cuda_dev), pool, cap, ws=ws)
            assert ws.status()[0] == 0
            assert torch.equal(dt.cpu(), t) and torch.equal(dl.cpu(), lens) and int(pool.free_count) == n
            assert torch.equal(df.cpu()[:n], f[:n])
            for x, y in zip((p.cu_tokens, p.positions, p.slots, p.seq_ids), ref):
                assert torch.equal(x.cpu(), y)
            dt.copy_(table), dl.copy_(old), df.copy_(free), pool.free_count.fill_(total - at)


def test_plan_empty(cuda_dev):
    i32 = dict(dtype=torch.int32, device=cuda_dev)
    pool = sa.PagePool.full(4, 16, cuda_dev)
    p = sa.plan_append(torch.zeros((0, 3), **i32), torch.zeros(0, **i32), torch.zeros(0, **i32), pool, 5)
    assert p.cu_tokens.tolist() == [0] and p.slots.tolist() == [-1] * 5 and int(pool.free_count) == 4
    lens = torch.zeros(2, **i32)
    p = sa.plan_append(torch.zeros((2, 3), **i32), lens, torch.zeros(2, **i32), pool, 0)
    assert p.cu_tokens.tolist() == [0, 0, 0] and p.slots.numel() == 0 and lens.tolist() == [0, 0]


@pytest.mark.parametrize("kind,want", [("pages", CAPACITY), ("tokens", CAPACITY), ("stack", CAPACITY),
                                       ("length", DEVICE_FAULT), ("too long", DEVICE_FAULT),
                                       ("new", DEVICE_FAULT), ("count", DEVICE_FAULT)])
def test_plan_that_does_not_fit_changes_nothing(cuda_dev, kind, want):
    table, old, new, free, count, total = _problem(11, 20, 16, 200)
    new[0], new[1], old[1] = 40, -1, 33
    held = int(((old + 15) // 16).sum())
    free = torch.arange(600, dtype=torch.int32)
    count, cap, stack = 300, int(new.clamp(min=0).sum()), free
    per = table.shape[1] + 4
    table = torch.nn.functional.pad(table, (0, 4), value=0).clamp(min=0)
    if kind == "pages":
        count = 0
        new[1] = 0
    elif kind == "tokens":
        cap -= 1
    elif kind == "stack":
        stack = free[:count]
    elif kind == "length":
        old[3] = -1
    elif kind == "too long":
        old[4], new[4] = per * 16, 1
    elif kind == "new":
        new[5] = -2
    elif kind == "count":
        count = 601
    assert held >= 0
    ws = sa.Workspace(cuda_dev)
    dt, dl, df = table.to(cuda_dev), old.to(cuda_dev), stack.clone().to(cuda_dev)
    pool = sa.PagePool(df, torch.tensor([count], dtype=torch.int32, device=cuda_dev), 600, 16)
    p = sa.plan_append(dt, dl, new.to(cuda_dev), pool, cap, ws=ws)
    st, det = ws.status()
    assert st == want, det
    assert torch.equal(dt.cpu(), table) and torch.equal(dl.cpu(), old) and torch.equal(df.cpu(), stack)
    assert int(pool.free_count) == count
    assert p.cu_tokens.abs().sum() == 0 and bool((p.slots == -1).all()) and bool((p.seq_ids == -1).all())


def test_plan_records_bad_pages(cuda_dev):
    """A bad page on the stack or in the table: its tokens get slot -1, the others their place."""
    table = torch.tensor([[3, -1, -1], [99, -1, -1]], dtype=torch.int32, device=cuda_dev)
    lens = torch.tensor([14, 2], dtype=torch.int32, device=cuda_dev)
    new = torch.tensor([20, 1], dtype=torch.int32, device=cuda_dev)
    pool = sa.PagePool(torch.tensor([6, 5, -4, 2], dtype=torch.int32, device=cuda_dev),
                       torch.tensor([4], dtype=torch.int32, device=cuda_dev), 8, 16)
    ws = sa.Workspace(cuda_dev)
    p = sa.plan_append(table, lens, new, pool, 21, ws=ws)
    assert ws.status()[0] == DEVICE_FAULT
    assert table.tolist() == [[3, 2, -1], [99, -1, -1]]
    assert p.slots.tolist() == [62, 63] + list(range(32, 48)) + [-1, -1] + [-1]


# ---------------------------------------------------------------------------
# norm + rotary append
# ---------------------------------------------------------------------------
def _inputs(seed, T, hq, hkv, d, page, packed=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, hq + 2 * hkv, d, generator=g) * (0.3 + torch.rand(hq + 2 * hkv, 1, generator=g))).bfloat16()
    pages = T // page + 3
    slots = torch.randperm(pages * page, generator=g)[:T]
    if T > 3:
        slots[T // 2] = -1
    pos = torch.randint(0, 1 << 20, (T,), generator=g).int()
    w = (1 + 0.2 * torch.randn(2, d, generator=g)).bfloat16()
    return g, x, pages, slots, pos, w


def _check_rows(got, ref, where):
    """bf16 rows of fp32 arithmetic: half a step of bf16, and the fp32 chain (a
    norm of d terms and a rotation: fewer than 64 roundings of 2^-24, relative
    to the row's largest element)."""
    got = got.double().cpu()
    lim = R.BF16_HALF * ref.abs() + 64 * 2.0 ** -24 * ref.abs().amax(-1, keepdim=True)
    assert bool(((got - ref).abs() <= lim).all()), (where, float(((got - ref).abs() - lim).max()))


CASES = [  # T, Hq, Hkv, d, page, rot, interleaved, norm
    (1, 4, 4, 64, 16, 64, False, True), (1, 64, 8, 128, 16, 128, False, True), (5, 32, 8, 128, 64, 128, True, True),
    (3, 5, 1, 128, 16, 64, False, True), (17, 12, 3, 64, 16, 32, True, False), (33, 8, 2, 128, 64, 0, False, True),
    (700, 7, 3, 128, 16, 128, False, False), (301, 3, 2, 64, 64, 48, False, True), (2, 1, 1, 128, 16, 16, True, True),
    (9999, 5, 3, 64, 64, 64, False, True), (9601, 4, 9, 128, 16, 32, True, True), (2, 2, 300, 128, 64, 128, False, True)]


@pytest.mark.parametrize("T,hq,hkv,d,page,rot,il,norm", CASES)
@pytest.mark.parametrize("wtype", [torch.bfloat16, torch.float32])
def test_append_bf16_pages(cuda_dev, T, hq, hkv, d, page, rot, il, norm, wtype):
    g, x, pages, slots, pos, w = _inputs(T + hq, T, hq, hkv, d, page)
    inv = (10000.0 ** (-torch.arange(0, rot, 2).double() / max(rot, 1))).float()
    w = w.to(wtype)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    kp = torch.randn(pages, hkv, page, d, generator=g).bfloat16()
    vp = torch.randn(pages, hkv, page, d, generator=g).bfloat16()
    c = sa.PagedCache(kp.to(cuda_dev), vp.to(cuda_dev), torch.zeros(1, 1, dtype=torch.int32, device=cuda_dev),
                      torch.zeros(1, dtype=torch.int32, device=cuda_dev))
    xd = x.to(cuda_dev)
    ws = sa.Workspace(cuda_dev)
    out = sa.rope_append(c, xd[:, :hq], xd[:, hq:hq + hkv], xd[:, hq + hkv:], pos.to(cuda_dev), slots.to(cuda_dev),
                         inv.to(cuda_dev) if rot else None, q_weight=w[0].to(cuda_dev) if norm else None,
                         k_weight=w[1].to(cuda_dev) if norm else None, eps=1e-5, interleaved=il, ws=ws)
    assert ws.status()[0] == 0
    assert torch.equal(xd.cpu(), x)                       # the projections are left as they were
    _check_rows(out, R.norm_rope(q, w[0] if norm else None, 1e-5, pos, inv, il), "q")
    ok = slots >= 0
    kr = R.norm_rope(k, w[1] if norm else None, 1e-5, pos, inv, il)
    pg, off = slots[ok] // page, slots[ok] % page
    gk, gv = c.k.cpu(), c.v.cpu()
    _check_rows(gk[pg, :, off], kr[ok], "k")
    assert torch.equal(gv[pg, :, off], v[ok])
    # every other slot is left as it was
    kp[pg, :, off], vp[pg, :, off] = gk[pg, :, off], gv[pg, :, off]
    assert torch.equal(gk, kp) and torch.equal(gv, vp)


@pytest.mark.parametrize("T,hq,hkv,d,page,rot,il,norm", CASES)
def test_append_4bit_pages_exactly(cuda_dev, T, hq, hkv, d, page, rot, il, norm):
    """The stored bytes are those of the 64-bit definition, bit for bit."""
    g, x, pages, slots, pos, w = _inputs(3 * T + hq, T, hq, hkv, d, page)
    inv = (500000.0 ** (-torch.arange(0, rot, 2).double() / max(rot, 1))).float()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    kv = R.random_records(g, pages, hkv, page, d)
    c = sa.PagedCache4(kv.to(cuda_dev), torch.zeros(1, 1, dtype=torch.int32, device=cuda_dev),
                       torch.zeros(1, dtype=torch.int32, device=cuda_dev))
    xd = x.to(cuda_dev)
    ws = sa.Workspace(cuda_dev)
    out = sa.rope_append(c, xd[:, :hq], xd[:, hq:hq + hkv], xd[:, hq + hkv:], pos.to(cuda_dev), slots.to(cuda_dev),
                         inv.to(cuda_dev) if rot else None, q_weight=w[0].to(cuda_dev) if norm else None,
                         k_weight=w[1].to(cuda_dev) if norm else None, interleaved=il, ws=ws)
    assert ws.status()[0] == 0
    _check_rows(out, R.norm_rope(q, w[0] if norm else None, 1e-6, pos, inv, il), "q")
    ok = slots >= 0
    rec = R.records(R.norm_rope(k, w[1] if norm else None, 1e-6, pos, inv, il), v.double())
    kv[slots[ok] // page, :, slots[ok] % page] = rec[ok]
    assert torch.equal(c.kv.cpu(), kv)


@pytest.mark.parametrize("d", [64, 128])
def test_4bit_rows_that_are_special(cuda_dev, d):
    """Constant rows, ties between codes, huge and tiny ones, infinities and NaN."""
    rows = torch.zeros(12, d)
    rows[0] = -3.5                                                  # no range: scale 0
    rows[1] = torch.arange(d) % 2 * 1.0                             # two values
    rows[2] = torch.tensor([0, 0.5, 1.5, 2.5, 3.5, 13.5, 14.5, 15.0]).repeat(d // 8)   # ties
    rows[3] = torch.linspace(-1, 1, d) * 3e38
    rows[4] = torch.linspace(-1, 1, d) * 1e-38                      # near the smallest normal numbers
    rows[5] = torch.linspace(1000, 1001, d)                         # far from zero
    rows[6, 3] = float("inf")
    rows[7, d - 1] = float("-inf")
    rows[8, d // 2] = float("nan")
    rows[9] = float("nan")
    rows[10] = -torch.arange(d).float()
    rows[11, 0] = 1e-30
    rows[11, d - 1] = -1.0
    x = rows.bfloat16()[:, None]
    T = len(rows)
    c = sa.PagedCache4.empty(1, 1, 16, d, torch.zeros(1, 1, dtype=torch.int32, device=cuda_dev),
                             torch.zeros(1, dtype=torch.int32, device=cuda_dev))
    xd = x.to(cuda_dev)
    sa.rope_append(c, xd, xd, xd, torch.zeros(T, dtype=torch.int32, device=cuda_dev),
                   torch.arange(T, device=cuda_dev))
    got, ref = c.kv.cpu()[0, 0, :T], R.records(x.double(), x.double())[:, 0]
    # a NaN parameter is a NaN, whatever its bits
    gp, rp = got[:, d:].contiguous().view(torch.bfloat16), ref[:, d:].contiguous().view(torch.bfloat16)
    assert torch.equal(got[:, :d], ref[:, :d])
    assert torch.equal(torch.isnan(gp), torch.isnan(rp)) and torch.equal(gp[~torch.isnan(gp)], rp[~torch.isnan(rp)])
    k, v = sa.expand_kv4(c, torch.zeros(1, dtype=torch.int32, device=cuda_dev))
    rk, rv, _ = R.values(ref)
    for a, b in ((k, rk), (v, rv)):
        a = a.cpu()[0, 0, :T].double()
        assert torch.equal(torch.isnan(a), torch.isnan(b))
        f = ~torch.isnan(b)
        # bf16 of zero + scale code by way of fp32: half a step, and 2^-24
        assert bool(((a - b)[f].abs() <= (R.BF16_HALF + 2.0 ** -23) * b[f].abs() + 1e-45).all())


@pytest.mark.parametrize("d,eps", [(64, 0.0), (128, 0.0), (128, 1e-6), (128, 1e30)])
def test_4bit_keys_of_every_size(cuda_dev, d, eps):
    """Keys whose squares overflow or vanish in fp32 still store the bytes of the 64-bit definition."""
    g = torch.Generator().manual_seed(int(d + 1e3 * min(eps, 1)))
    size = 10.0 ** torch.arange(-36, 37, 4).double()
    T = len(size)
    x = (torch.randn(T, 2, d, generator=g).double() * size[:, None, None]).bfloat16()
    x[3, 1, 5:] = 0                                                  # a row with few elements
    w = (1 + 0.2 * torch.randn(d, generator=g)).bfloat16()
    pos = torch.arange(T).int() * 1000
    inv = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float()
    c = sa.PagedCache4.empty(2, 2, 64, d, torch.zeros(1, 1, dtype=torch.int32, device=cuda_dev),
                             torch.zeros(1, dtype=torch.int32, device=cuda_dev))
    xd = x.to(cuda_dev)
    sa.rope_append(c, xd, xd, xd, pos.to(cuda_dev), torch.arange(T, device=cuda_dev), inv.to(cuda_dev),
                   k_weight=w.to(cuda_dev), eps=eps)
    # (eps reaches the library as fp32)
    ref = R.records(R.norm_rope(x, w, float(torch.tensor(eps, dtype=torch.float32)), pos, inv, False), x.double())
    assert torch.equal(c.kv.cpu()[0, :, :T].transpose(0, 1), ref)


def test_append_in_place_strided_and_on_a_stream(cuda_dev):
    """q_out = q inside a packed projection, on a side stream, equals the plain call."""
    T, hq, hkv, d = 37, 8, 2, 128
    g, x, pages, slots, pos, w = _inputs(5, T, hq, hkv, d, 16)
    inv = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float().to(cuda_dev)
    mk = lambda: sa.PagedCache4.empty(pages, hkv, 16, d, torch.zeros(1, 1, dtype=torch.int32, device=cuda_dev),
                                      torch.zeros(1, dtype=torch.int32, device=cuda_dev))
    a, b, c = mk(), mk(), mk()
    xd, pd, sd, wd = x.to(cuda_dev), pos.to(cuda_dev), slots.to(cuda_dev), w.to(cuda_dev)
    kw = dict(q_weight=wd[0], k_weight=wd[1])
    ref = sa.rope_append(a, xd[:, :hq], xd[:, hq:hq + hkv], xd[:, hq + hkv:], pd, sd, inv, **kw)
    y = xd.clone()
    s = torch.cuda.Stream(cuda_dev)
    s.wait_stream(torch.cuda.current_stream(cuda_dev))
    q = y[:, :hq]
    out = sa.rope_append(b, q, y[:, hq:hq + hkv], y[:, hq + hkv:], pd, sd, inv, q_out=q, stream=s, **kw)
    torch.cuda.current_stream(cuda_dev).wait_stream(s)
    assert out is q and torch.equal(q, ref) and torch.equal(y[:, hq:], xd[:, hq:]) and torch.equal(a.kv, b.kv)
    # heads and tokens apart: copied by the binding
    z = torch.zeros(T, 2 * hq, d, dtype=torch.bfloat16, device=cuda_dev)
    z[:, ::2] = xd[:, :hq]
    out = sa.rope_append(c, z[:, ::2], xd[:, hq:hq + hkv].contiguous(), xd[:, hq + hkv:], pd, sd, inv, **kw)
    assert torch.equal(out, ref) and torch.equal(a.kv, c.kv)


def test_append_records_bad_slots(cuda_dev):
    T, d = 6, 64
    x = torch.randn(T, 3, d, device=cuda_dev).bfloat16()
    c = sa.PagedCache4.empty(2, 1, 16, d, torch.zeros(1, 1, dtype=torch.int32, device=cuda_dev),
                             torch.zeros(1, dtype=torch.int32, device=cuda_dev))
    slots = torch.tensor([0, 32, -2, 31, 1 << 40, -1], device=cuda_dev)
    ws = sa.Workspace(cuda_dev)
    q = sa.rope_append(c, x[:, :1], x[:, 1:2], x[:, 2:], torch.zeros(T, dtype=torch.int32, device=cuda_dev), slots,
                       ws=ws)
    st, det = ws.status()
    assert st == DEVICE_FAULT and det[1] == 12
    assert torch.equal(q, x[:, :1])
    used = c.kv.view(32, d + 16).any(-1)
    assert used.nonzero().flatten().tolist() == [0, 31]


@pytest.mark.parametrize("d,page,hkv", [(64, 16, 3), (128, 64, 2), (128, 16, 1)])
def test_expand_pages(cuda_dev, d, page, hkv):
    g = torch.Generator().manual_seed(d + page)
    kv = R.random_records(g, 9, hkv, page, d)
    c = sa.PagedCache4(kv.to(cuda_dev), torch.zeros(1, 1, dtype=torch.int32, device=cuda_dev),
                       torch.zeros(1, dtype=torch.int32, device=cuda_dev))
    pages = torch.tensor([8, 0, 3, -1, 3, 9, -5], dtype=torch.int32)
    k0 = torch.randn(7, hkv, page, d, generator=g).bfloat16()
    k, v = k0.to(cuda_dev), (2 * k0).to(cuda_dev)
    ws = sa.Workspace(cuda_dev)
    rk, rv = sa.expand_kv4(c, pages.to(cuda_dev), k, v, ws=ws)
    st, det = ws.status()
    assert rk is k and rv is v and st == DEVICE_FAULT and det[2] in (9, -5)
    ek, ev, _ = R.values(kv[pages.clamp(0, 8).long()])
    for got, ref, was in ((k.cpu(), ek, k0), (v.cpu(), ev, 2 * k0)):
        for i, p in enumerate(pages.tolist()):
            if 0 <= p < 9:
                lim = (R.BF16_HALF + 2.0 ** -23) * ref[i].abs()
                assert bool(((got[i].double() - ref[i]).abs() <= lim).all())
            else:
                assert torch.equal(got[i], was[i])
    k, v = sa.expand_kv4(c, torch.zeros(0, dtype=torch.int32, device=cuda_dev))
    assert k.shape == (0, hkv, page, d)
