"""Cases of the serving-step operators around the paged KV cache: planning the
pages of a step (block tables and slots), writing its keys and values (per-head
norm, rotary positions, the store into a bf16 or 4-bit cache), reading pages of
a 4-bit cache back to bf16, and sparse decode attention over a 4-bit cache.

``run`` computes a case either through the package's entry points (``own``) or
in plain torch operations.  The 4-bit cache keeps, per (page, kv head, token),
one record of ``d + 16`` bytes:

  bytes [0, d/2)      codes of the key, channel 2j in the low nibble of byte j
  bytes [d/2, d)      codes of the value, likewise
  bytes [d, d + 16)   8 bf16 numbers: {scale, zero} of the key's first and
                      second half of channels, then of the value's halves

and a code c of a half stands for zero + scale * c.  A half x is stored as
zero = bf16(min x), scale = bf16((max x - min x) / 15) (each through fp32) and
c = the nearest whole number to (x - zero) / scale, ties to even, in [0, 15].
"""
import math

import torch

own = False

DEV = "cuda"

# A sequence's list entry, a page table entry and a position are int32, a slot
# (physical page * page size + offset, -1 = store nothing) is int64.


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token for each of 32 running sequences: the call of every decode step
        dict(name="plan, a decode step", op="plan", seqs=32, page=16, max_len=65536, tokens=32, kind="step"),
        # continuous batching: prompts in chunks beside running, idle and finished sequences
        dict(name="plan, chunked prompts", op="plan", seqs=256, page=64, max_len=32768, tokens=131072, kind="mixed"),
        # keys and values of one decode step, into bf16 pages
        dict(name="append, a decode step", op="append", tokens=32, seqs=32, q_heads=32, kv_heads=8, dim=128,
             page=16, rot=128, interleaved=False, norm=True, bits=16),
        # a 32768-token prompt's prefill, one layer
        dict(name="append, a prompt", op="append", tokens=32768, seqs=1, q_heads=32, kv_heads=4, dim=128,
             page=64, rot=128, interleaved=False, norm=True, bits=16),
        # one step of the long-context masked decode (64/8 heads), into 4-bit pages, read back
        dict(name="append 4-bit, a decode step", op="append", tokens=4, seqs=4, q_heads=64, kv_heads=8, dim=128,
             page=16, rot=128, interleaved=False, norm=True, bits=4),
        # chunked prompts of several sequences into 4-bit pages, read back for a prefill on bf16 pages
        dict(name="append 4-bit, prompts", op="append", tokens=16391, seqs=7, q_heads=32, kv_heads=8, dim=128,
             page=16, rot=64, interleaved=True, norm=True, bits=4),
        # a short cached context expanded before its next chunk is prefilled
        dict(name="expand, a short context", op="expand", pages=129, kv_heads=8, dim=128, page=16),
        # a 131072-token context expanded for the block-sparse prefill (64-token pages)
        dict(name="expand, a long context", op="expand", pages=2048, kv_heads=4, dim=128, page=64),
        # the smallest decode: one sequence, 4 heads, 256 of 4096 tokens, fp32 queries
        dict(name="decode 4-bit, tiny", op="tokens", seqs=1, q_heads=4, kv_heads=4, dim=64, page=16, length=4096,
             k=256, f32=True),
        # a reuse layer of a large batch: each head's own 4096 of 65536 tokens
        dict(name="decode 4-bit, token lists", op="tokens", seqs=32, q_heads=32, kv_heads=8, dim=128, page=16,
             length=65536, k=4096, f32=False),
        # focus, local and streaming spans over 131072 tokens, one step
        dict(name="decode 4-bit, masked", op="blocks", seqs=4, q_heads=64, kv_heads=8, dim=128, page=16,
             length=131072, kind="masked", f32=False),
        # a global step: every page of 32 sequences of up to 16384 tokens
        dict(name="decode 4-bit, whole context", op="blocks", seqs=32, q_heads=32, kv_heads=8, dim=128, page=64,
             length=16384, kind="global", f32=False),
    ]


_HEADS = [(4, 4), (8, 2), (8, 8), (12, 3), (16, 2), (32, 4), (32, 8), (64, 8), (16, 1), (5, 1)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "expand", "tokens", "tokens", "blocks", "blocks"])
    if op == "plan":
        kind = rng.choice(["step", "mixed"])
        seqs = _log(rng, 1, 512)
        return dict(op=op, seqs=seqs, page=rng.choice([16, 64]), max_len=_log(rng, 256, 32768),
                    tokens=seqs + rng.randrange(9) if kind == "step" else _log(rng, 64, 131072), kind=kind)
    hq, hkv = rng.choice(_HEADS)
    dim, page = rng.choice([64, 128, 128]), rng.choice([16, 64])
    if op == "append":
        tokens = _log(rng, 1, max(2, 32768 * 40 // (hq + 2 * hkv) // 2))
        return dict(op=op, tokens=tokens, seqs=rng.randint(1, min(tokens, 64)), q_heads=hq, kv_heads=hkv, dim=dim,
                    page=page, rot=rng.choice([dim, dim, dim // 2, 0]), interleaved=rng.random() < 0.4,
                    norm=rng.random() < 0.8, bits=rng.choice([16, 4]))
    if op == "expand":
        return dict(op=op, pages=_log(rng, 1, 524288 // (hkv * page)), kv_heads=hkv, dim=dim, page=page)
    if op == "tokens":
        k = _log(rng, 1, 4096)
        seqs = max(1, min(_log(rng, 1, 64), 4194304 // (hq * k)))
        length = _log(rng, max(64, k), max(65, min(131072, 8388608 // (hkv * seqs))))
        return dict(op=op, seqs=seqs, q_heads=hq, kv_heads=hkv, dim=dim, page=page, length=length, k=k,
                    f32=rng.random() < 0.3)
    seqs = _log(rng, 1, 64)
    length = _log(rng, 1, max(2, min(131072, 4194304 // (hkv * seqs))))
    return dict(op=op, seqs=seqs, q_heads=hq, kv_heads=hkv, dim=dim, page=page, length=length,
                kind=rng.choice(["masked", "global"]), f32=rng.random() < 0.3)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed, device=None):
    g = torch.Generator(device=device or DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=g.device)


def _ints(g, lo, hi, *shape):
    """Whole numbers in [lo, hi), on the CPU."""
    return torch.randint(lo, hi, shape, generator=g)


def _quantized(g, rows, dim):
    """Records [rows][dim + 16] of Gaussian keys (with a mean per channel, as
    keys have) and values."""
    out = torch.empty(rows, dim + 16, dtype=torch.uint8, device=DEV)
    mean = _randn(g, dim)
    for a in range(0, rows, 1 << 20):
        b = min(rows, a + (1 << 20))
        x = torch.stack([_randn(g, b - a, dim) + mean, _randn(g, b - a, dim)], 1)
        h = x.view(b - a, 4, dim // 2)
        lo = h.amin(-1, keepdim=True)
        par = torch.cat([(h.amax(-1, keepdim=True) - lo) / 15, lo], -1).bfloat16()
        c = ((h - par[..., 1:].float()) / par[..., :1].float()).round().clamp(0, 15).to(torch.uint8)
        c = c.view(b - a, dim, 2)
        out[a:b, :dim] = c[..., 0] | (c[..., 1] << 4)
        out[a:b, dim:] = par.reshape(b - a, 8).view(torch.uint8)
    return out


def _lengths(g, seqs, most, least=1):
    """Ragged lengths, the first the longest; log-spread below it."""
    u = torch.rand(seqs, generator=g, dtype=torch.float64)
    n = (most * torch.exp(-0.7 * u)).long().clamp(least, most)
    n[0] = most
    return n


def _cache4(case, seed):
    """A 4-bit pool, a shuffled page table and ragged lengths."""
    g, c = _gen(seed), _gen(seed + 1, "cpu")
    B, P, L = case["seqs"], case["page"], case["length"]
    per = -(-L // P)
    pages = B * per + 3
    kv = _quantized(g, pages * case["kv_heads"] * P, case["dim"]).view(pages, case["kv_heads"], P, case["dim"] + 16)
    table = torch.randperm(pages, generator=c)[: B * per].view(B, per).int().to(DEV)
    lens = _lengths(c, B, L)
    if B > 3:
        lens[B - 2] = 0  # a slot of the batch with nothing in it
    q = _randn(g, B, case["q_heads"], case["dim"])
    q = q if case["f32"] else q.bfloat16()
    return g, c, dict(op=case["op"], kv=kv, table=table, lens=lens.int().to(DEV), q=q, dim=case["dim"], page=P), lens


def _plan_state(case, seed):
    c = _gen(seed, "cpu")
    B, P, cap = case["seqs"], case["page"], case["tokens"]
    per = -(-(2 * case["max_len"]) // P)
    old = _lengths(c, B, case["max_len"], 0)
    if case["kind"] == "step":
        new = torch.ones(B, dtype=torch.long)
    else:
        what = torch.rand(B, generator=c)
        new = (torch.rand(B, generator=c).double() * min(case["max_len"], 2 * cap // B + 1)).long()
        new[what < 0.4] = 1                       # running
        new[what < 0.2] = 0                       # idle
        new[what < 0.1] = -1                      # finished
        old[(what > 0.7)] = 0                     # admitted in this step
        over = new.clamp(min=0).cumsum(0) > cap   # what does not fit the step waits
        new[over] = 0
    held = (old + P - 1) // P
    total = B * -(-case["max_len"] // P) + cap // P + B + 17
    perm = torch.randperm(total, generator=c).int()
    table = torch.full((B, per), -1, dtype=torch.int32)
    at = torch.arange(per).expand(B, per)
    mine = at < held[:, None]
    table[mine] = perm[: int(held.sum())]
    free = torch.full((total,), -1, dtype=torch.int32)
    count = total - int(held.sum())
    free[:count] = perm[int(held.sum()):]
    state = dict(op="plan", page=P, cap=cap, total=total, table=table.to(DEV), lens=old.int().to(DEV),
                 new=new.int().to(DEV), free=free.to(DEV), count=torch.tensor([count], dtype=torch.int32, device=DEV),
                 lens_out=torch.empty(B, dtype=torch.int32, device=DEV),
                 count_out=torch.empty(1, dtype=torch.int32, device=DEV))
    return state


def _append_state(case, seed):
    g, c = _gen(seed), _gen(seed + 1, "cpu")
    T, S, P, D = case["tokens"], case["seqs"], case["page"], case["dim"]
    hq, hkv = case["q_heads"], case["kv_heads"]
    # the projections' packed rows; each head of its own size, as real ones are
    qkv = (_randn(g, T, hq + 2 * hkv, D) * (0.5 + torch.rand(hq + 2 * hkv, 1, generator=g, device=DEV))).bfloat16()
    cut = torch.cat([torch.zeros(1).long(), (torch.randperm(T - 1, generator=c)[: S - 1] + 1).sort().values,
                     torch.tensor([T])])
    n = cut.diff()
    start = _ints(c, 0, 1 << 20, S)
    seq = torch.repeat_interleave(torch.arange(S), n)
    pos = start[seq] + torch.arange(T) - cut[seq]
    # pages of the sequences, from the one that holds each's first new token on
    first = start // P
    held = (start + n - 1) // P - first + 1
    base = torch.cat([torch.zeros(1).long(), held.cumsum(0)])
    pages = T // P + 2 * S + 1
    perm = torch.randperm(pages - 1, generator=c)
    slot = perm[base[seq] + pos // P - first[seq]] * P + pos % P
    if T > 8:
        slot[-(T // 64) or T:] = -1               # rows that only fill the batch up
    inv = (10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / max(1, case["rot"]))).float()
    w = (1 + 0.1 * _randn(g, 2, D)).bfloat16()
    state = dict(op="append", bits=case["bits"], page=P, dim=D, rot=case["rot"], interleaved=case["interleaved"],
                 q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], pos=pos.int().to(DEV),
                 slot=slot.to(DEV), inv=inv.to(DEV), wq=w[0] if case["norm"] else None,
                 wk=w[1] if case["norm"] else None, eps=1e-6)
    if case["bits"] == 16:
        state["kp"], state["vp"] = (_randn(g, pages, hkv, P, D).bfloat16() for _ in range(2))
    else:
        state["kv"] = _quantized(g, pages * hkv * P, D).view(pages, hkv, P, D + 16)
        state["pages"] = torch.randperm(pages, generator=c).int().to(DEV)
    state["table"] = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    state["lens"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return state


def _token_state(case, seed):
    g, c, state, lens = _cache4(case, seed)
    B, H, k = case["seqs"], case["q_heads"], case["k"]
    count = torch.minimum(torch.full((B, H), k), lens[:, None])
    # most heads keep k tokens, some fewer
    short = torch.rand(B, H, generator=c) < 0.1
    count = torch.where(short, (count * torch.rand(B, H, generator=c)).long(), count).to(DEV)
    i = torch.arange(k, device=DEV)
    n = count.clamp(min=1)[..., None]
    length = lens.to(DEV)[:, None, None]
    a, b = i * length // n, (i + 1) * length // n
    pick = a + ((b - a) * torch.rand(B, H, k, generator=g, device=DEV)).long().minimum((b - a - 1).clamp(min=0))
    state["idx"] = torch.where(i < count[..., None], pick, -1).int()
    state["count"] = count.int()
    return state


def _spans(kind, n, c, turn):
    """[start, end, rounded out to pages] of a mode of the decode."""
    if kind == "global":
        return [(0, n)]
    if turn % 3 == 0:      # focus: two chunks of 2048 tokens
        chunks = -(-n // 2048)
        at = torch.randperm(chunks, generator=c)[:2].sort().values.tolist()
        return [(2048 * x, min(n, 2048 * (x + 1))) for x in at]
    if turn % 3 == 1:      # local: the last 512 tokens
        return [(max(0, n - 512), n)]
    return [(0, min(4, n)), (max(4, n - 1024), n)] if n > 4 else [(0, n)]   # streaming


def _block_state(case, seed):
    g, c, state, lens = _cache4(case, seed)
    P, rows = case["page"], []
    for b, n in enumerate(lens.tolist()):
        parts, before = [], 0
        for s, e in _spans(case["kind"], n, c, b) if n else []:
            p = torch.arange(s // P, (e - 1) // P + 1) if e > s else torch.zeros(0).long()
            lo, hi = (s - p * P).clamp(min=0), (e - p * P).clamp(max=P)
            parts.append(torch.stack([p, lo, hi, before + (hi - lo).cumsum(0) - (hi - lo)], 1))
            before += max(0, e - s)
        rows.append(torch.cat(parts) if parts else torch.zeros(0, 4).long())
    most = max(1, max(len(r) for r in rows))
    blocks = torch.full((len(rows), most, 4), -1, dtype=torch.int32)
    for b, r in enumerate(rows):
        blocks[b, : len(r)] = r.int()
    state["blocks"] = blocks.to(DEV)
    state["count"] = torch.tensor([len(r) for r in rows], dtype=torch.int32, device=DEV)
    return state


def _expand_state(case, seed):
    g, c = _gen(seed), _gen(seed + 1, "cpu")
    n, hkv, P, D = case["pages"], case["kv_heads"], case["page"], case["dim"]
    pool = n + n // 2 + 3
    kv = _quantized(g, pool * hkv * P, D).view(pool, hkv, P, D + 16)
    return dict(op="expand", kv=kv, dim=D, pages=torch.randperm(pool, generator=c)[:n].int().to(DEV),
                table=torch.zeros(1, 1, dtype=torch.int32, device=DEV),
                lens=torch.zeros(1, dtype=torch.int32, device=DEV))


_STATES = {"plan": _plan_state, "append": _append_state, "tokens": _token_state, "blocks": _block_state,
           "expand": _expand_state}


def prepare(case, seed):
    return _STATES[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _values(rec, dim):
    """Records [..., dim + 16] -> fp32 (key, value) [..., dim] each."""
    c = rec[..., :dim]
    c = torch.stack([c & 15, c >> 4], -1).flatten(-2).unflatten(-1, (4, dim // 2))
    p = rec[..., dim:].contiguous().view(torch.bfloat16).float().unflatten(-1, (4, 2))
    x = torch.addcmul(p[..., 1:], p[..., :1], c.float()).flatten(-2)
    return x[..., :dim], x[..., dim:]


def _plain_plan(s):
    P, cap = s["page"], s["cap"]
    old, new, table, free = s["lens"].long(), s["new"].long(), s["table"], s["free"]
    gone, add = new < 0, new.clamp(min=0)
    held = (old + P - 1) // P
    lens = torch.where(gone, 0, old + add)
    need = torch.where(gone, 0, (lens + P - 1) // P - held)
    back = torch.where(gone, held, 0)
    # the pages of finished sequences go on top of the stack, in order ...
    p = torch.arange(table.shape[1], device=DEV)
    count = s["count"].long()
    put = count + (back.cumsum(0) - back)[:, None] + p
    put = torch.where(p < back[:, None], put, free.numel())
    stack = torch.cat([free, free.new_zeros(1)]).scatter(0, put.flatten(), table.flatten())[:-1]
    free = torch.where(torch.arange(free.numel(), device=DEV) < count + back.sum(), stack, free)
    # ... and the pages this step needs come off it, in order
    top = count + back.sum()
    take = (need.cumsum(0) - need)[:, None] + p - held[:, None]
    fresh = (p >= held[:, None]) & (p < (held + need)[:, None])
    table = torch.where(fresh, free[(top - 1 - take).clamp(0, free.numel() - 1)], table)
    ends = add.cumsum(0)
    cu = torch.cat([ends.new_zeros(1), ends])
    i = torch.arange(cap, device=DEV)
    real = i < cu[-1]
    seq = torch.searchsorted(ends, i, right=True).clamp(max=old.numel() - 1)
    pos = torch.where(real, old[seq] + i - cu[seq], 0)
    slot = torch.where(real, table[seq, pos // P].long() * P + pos % P, -1)
    return dict(table=table, lens=lens.int(), free=free, count=(top - need.sum()).int(), cu=cu.int(),
                positions=pos.int(), slots=slot, seqs=torch.where(real, seq, -1).int())


def _rope(x, angle, interleaved):
    """x [T][H][dim] with angle [T][rot / 2]: the first rot channels turned."""
    n = angle.shape[1]
    cos, sin = torch.cos(angle)[:, None].to(x.dtype), torch.sin(angle)[:, None].to(x.dtype)
    head, tail = x[..., : 2 * n], x[..., 2 * n:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head[..., :n], head[..., n:]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([head, tail], -1)


def _normed(x, w, eps):
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.to(x.dtype)


def _records(k, v):
    """fp64 rows [T][H][dim] of keys and values -> records [T][H][dim + 16]."""
    dim = k.shape[-1]
    h = torch.cat([k, v], -1).unflatten(-1, (4, dim // 2))
    lo = h.amin(-1, keepdim=True)
    par = torch.cat([(h.amax(-1, keepdim=True) - lo) / 15, lo], -1).float().bfloat16()
    scale, zero = par[..., :1].double(), par[..., 1:].double()
    c = torch.where(scale > 0, (h - zero) / torch.where(scale > 0, scale, 1), 0).round().clamp(0, 15).to(torch.uint8)
    c = c.flatten(-2).unflatten(-1, (dim, 2))
    return torch.cat([c[..., 0] | (c[..., 1] << 4), par.flatten(-2).contiguous().view(torch.uint8)], -1)


def _store(pool, page, off, keep, rows):
    """Rows into pool [pages][heads][page size][...]; those not kept write the
    pool's last row over itself (its last page is no sequence's)."""
    page, off = torch.where(keep, page, pool.shape[0] - 1), torch.where(keep, off, pool.shape[2] - 1)
    pool[page, :, off] = torch.where(keep[:, None, None], rows, pool[-1, :, -1])


def _plain_append(s):
    angle = s["pos"].double()[:, None] * s["inv"].double()
    q = _rope(_normed(s["q"].float(), s["wq"], s["eps"]), angle, s["interleaved"]).bfloat16()
    keep = s["slot"] >= 0
    slot = torch.where(keep, s["slot"], 0)
    page, off = slot // s["page"], slot % s["page"]
    # a 4-bit code next to a border hangs on the last bits: in 64
    k = s["k"].float() if s["bits"] == 16 else s["k"].double()
    k = _rope(_normed(k, s["wk"], s["eps"]), angle, s["interleaved"])
    if s["bits"] == 16:
        _store(s["kp"], page, off, keep, k.bfloat16())
        _store(s["vp"], page, off, keep, s["v"])
        return q, s["kp"], s["vp"]
    _store(s["kv"], page, off, keep, _records(k, s["v"].double()))
    key, value = _values(s["kv"][s["pages"].long()], s["dim"])
    return q, key.bfloat16(), value.bfloat16()


def _plain_expand(s):
    key, value = _values(s["kv"][s["pages"].long()], s["dim"])
    return key.bfloat16(), value.bfloat16()


def _softmax_sum(score, real, value):
    """Softmax over the last axis of score where real, times value [..., n, dim]."""
    score = torch.where(real, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e.unsqueeze(-2), value).squeeze(-2) / torch.where(total > 0, total, 1.0)
    return out.bfloat16(), (torch.log(total) + top).squeeze(-1)


def _plain_tokens(s):
    B, H, D = s["q"].shape
    hkv, P = s["kv"].shape[1], s["page"]
    real = torch.arange(s["idx"].shape[-1], device=DEV) < s["count"][..., None]
    t = torch.where(real, s["idx"], 0).long()
    page = torch.gather(s["table"].long()[:, None].expand(B, H, -1), 2, t // P)
    group = (torch.arange(H, device=DEV) // (H // hkv))[None, :, None]
    key, value = _values(s["kv"][page, group, t % P], D)
    score = torch.matmul(key, s["q"].float().unsqueeze(-1)).squeeze(-1) / math.sqrt(D)
    return _softmax_sum(score, real, value)


def _plain_blocks(s):
    B, H, D = s["q"].shape
    hkv, P = s["kv"].shape[1], s["page"]
    e = s["blocks"].long()
    n = e.shape[1]
    off = torch.arange(P, device=DEV)
    listed_ = torch.arange(n, device=DEV) < s["count"][:, None]
    real = listed_[..., None] & (off >= e[..., 1:2]) & (off < e[..., 2:3])
    page = torch.gather(s["table"].long(), 1, torch.where(listed_, e[..., 0], 0))
    rec = s["kv"][page].transpose(1, 2).reshape(B, hkv, n * P, D + 16)
    key, value = _values(rec, D)
    q = s["q"].float().view(B, hkv, H // hkv, D)
    score = torch.matmul(q, key.transpose(-1, -2)) / math.sqrt(D)
    real = real.view(B, 1, 1, n * P)
    score = torch.where(real, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    total = w.sum(-1, keepdim=True)
    out = torch.matmul(w, value) / torch.where(total > 0, total, 1.0)
    return out.reshape(B, H, D).bfloat16(), (torch.log(total) + top).reshape(B, H)


_PLAIN = {"plan": _plain_plan, "append": _plain_append, "expand": _plain_expand, "tokens": _plain_tokens,
          "blocks": _plain_blocks}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(s):
    import sparse_attention_aware_b200 as sa
    op = s["op"]
    if op == "plan":
        pool = sa.PagePool(s["free"], s["count"], s["total"], s["page"])
        p = sa.plan_append(s["table"], s["lens"], s["new"], pool, s["cap"], seq_lens_out=s["lens_out"],
                           free_count_out=s["count_out"])
        return dict(table=s["table"], lens=s["lens_out"], free=s["free"], count=s["count_out"], cu=p.cu_tokens,
                    positions=p.positions, slots=p.slots, seqs=p.seq_ids)
    if op == "append" and s["bits"] == 16:
        cache = sa.PagedCache(s["kp"], s["vp"], s["table"], s["lens"])
        q = sa.rope_append(cache, s["q"], s["k"], s["v"], s["pos"], s["slot"], s["inv"], q_weight=s["wq"],
                           k_weight=s["wk"], eps=s["eps"], interleaved=s["interleaved"])
        return q, s["kp"], s["vp"]
    cache = sa.PagedCache4(s["kv"], s["table"], s["lens"])
    if op == "append":
        q = sa.rope_append(cache, s["q"], s["k"], s["v"], s["pos"], s["slot"], s["inv"], q_weight=s["wq"],
                           k_weight=s["wk"], eps=s["eps"], interleaved=s["interleaved"])
        return (q,) + tuple(sa.expand_kv4(cache, s["pages"]))
    if op == "expand":
        return tuple(sa.expand_kv4(cache, s["pages"]))
    if op == "tokens":
        sel = sa.TokenSelection(s["idx"], s["count"])
    else:
        sel = sa.BlockSelection(s["blocks"], s["count"])
    return sa.sparse_decode_attn(cache, s["q"], sel, num_splits=0)


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, P = case["op"], case["page"]
    if op == "plan":
        # lengths in and out, the prefix sums, a table entry and a stack entry for
        # each fresh page, and a position, a slot and a sequence for each token
        B, n = case["seqs"], case["tokens"]
        return {"bytes": 16 * B + 16 * n + 8 * (n // P), "flops": 0}
    hkv, D = case["kv_heads"], case["dim"]
    if op == "append":
        T, hq = case["tokens"], case["q_heads"]
        row = 2 * D if case["bits"] == 16 else (D + 16) / 2
        read = T * (hq + 2 * hkv) * 2 * D
        wrote = T * hq * 2 * D + T * 2 * hkv * row
        back = 0 if case["bits"] == 16 else T * hkv * ((D + 16) + 4 * D)
        return {"bytes": read + wrote + back + 12 * T, "flops": 10 * T * (hq + hkv) * D}
    if op == "expand":
        rows = case["pages"] * hkv * P
        return {"bytes": rows * (D + 16 + 4 * D), "flops": 4 * rows * D}
    B, H, L = case["seqs"], case["q_heads"], case["length"]
    # lengths are max * exp(-0.7 u): their mean
    mean = L if B == 1 else L * (1 - math.exp(-0.7)) / 0.7
    if op == "tokens":
        n = min(case["k"], mean)
        group = H // hkv
        rows = B * hkv * mean * (1 - (1 - n / mean) ** group)    # a row that several heads of a group keep: once
        each = B * H * n
        extra = 4 * each
    else:
        n = mean if case["kind"] == "global" else min(mean, (4096 + 512 + 1028) / 3)
        rows, each = B * hkv * n, B * H * n
        extra = 16 * B * n / P + 4 * B * n / P
    return {"bytes": rows * (D + 16) + extra + B * H * D * (4 if case["f32"] else 2) + B * H * (2 * D + 4),
            "flops": 4 * each * D}


# ---------------------------------------------------------------------------
# in 64 bits, from the definitions
# ---------------------------------------------------------------------------
def _read64(rec, dim):
    """(key, value) of records, one channel pair of a byte at a time, in fp64."""
    out = []
    for side in range(2):
        byte = rec[..., side * dim // 2:(side + 1) * dim // 2].long()
        code = torch.empty(*byte.shape[:-1], dim, dtype=torch.float64, device=rec.device)
        code[..., 0::2], code[..., 1::2] = (byte % 16).double(), (byte // 16).double()
        raw = rec[..., dim + 8 * side: dim + 8 * side + 8].long()
        bits = (raw[..., 0::2] + 256 * raw[..., 1::2]) * 65536          # bf16 = the high half of an fp32
        par = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).int().view(torch.float32).double()
        for half in range(2):
            c = slice(half * dim // 2, (half + 1) * dim // 2)
            code[..., c] = code[..., c] * par[..., 2 * half, None] + par[..., 2 * half + 1, None]
        out.append(code)
    return out


def _turn64(x, w, eps, pos, inv, interleaved):
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + eps).sqrt() * w.double()
    n = inv.numel()
    if not n:
        return x
    e = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                    pos.double()[:, None] * inv.double()[None])[:, None]
    x = x.clone()
    if interleaved:
        z = torch.complex(x[..., 0:2 * n:2], x[..., 1:2 * n:2]) * e
        x[..., 0:2 * n:2], x[..., 1:2 * n:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :n], x[..., n:2 * n]) * e
        x[..., :n], x[..., n:2 * n] = z.real, z.imag
    return x


def _stored64(x):
    """What a 4-bit row gives back: zero + scale * c, c counted up border by border."""
    out = torch.empty_like(x)
    half = x.shape[-1] // 2
    for a in (0, half):
        y = x[..., a:a + half]
        lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
        zero, scale = lo.float().bfloat16().double(), ((hi - lo) / 15).float().bfloat16().double()
        d, c = y - zero, torch.zeros_like(y)
        for j in range(15):
            border = (j + 0.5) * scale
            c += (d > border) | ((d == border) & (j % 2 == 1) & (scale > 0))
        out[..., a:a + half] = zero + scale * torch.where(scale > 0, c, 0)
    return out


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None
    s = prepare(case, seed)
    D = case["dim"]
    if op == "expand":
        return tuple(_read64(s["kv"][s["pages"].long()], D))
    if op == "append":
        q = _turn64(s["q"], s["wq"], s["eps"], s["pos"], s["inv"], s["interleaved"])
        k = _turn64(s["k"], s["wk"], s["eps"], s["pos"], s["inv"], s["interleaved"])
        v = s["v"].double()
        ok = s["slot"] >= 0
        page, off = s["slot"][ok] // s["page"], s["slot"][ok] % s["page"]
        if s["bits"] == 16:
            pools = [s["kp"].double(), s["vp"].double()]
            rows = [k, v]
        else:
            pools = _read64(s["kv"], D)
            rows = [_stored64(k), _stored64(v)]
        for pool, r in zip(pools, rows):
            pool[page, :, off] = r[ok]
        if s["bits"] == 4:
            pools = [p[s["pages"].long()] for p in pools]
        return (q, *pools)
    B, H, _ = s["q"].shape
    hkv, P = s["kv"].shape[1], s["page"]
    out = torch.zeros(B, H, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device=DEV)
    table = s["table"].long()
    for b in range(B):
        for g in range(hkv):
            heads = range(g * (H // hkv), (g + 1) * (H // hkv))
            if op == "blocks":
                t = _tokens_of(s["blocks"][b, : int(s["count"][b])].long(), P)
                if not t.numel():
                    continue
                k, v = _read64(s["kv"][table[b, t // P], g, t % P], D)
            for h in heads:
                if op == "tokens":
                    t = s["idx"][b, h, : int(s["count"][b, h])].long()
                    if not t.numel():
                        continue
                    k, v = _read64(s["kv"][table[b, t // P], g, t % P], D)
                z = (k @ s["q"][b, h].double()) / math.sqrt(D)
                lse[b, h] = torch.logsumexp(z, 0)
                out[b, h] = torch.exp(z - lse[b, h]) @ v
    return out, lse


def _tokens_of(e, P):
    """The tokens of list entries, in order."""
    if not len(e):
        return torch.zeros(0, dtype=torch.long, device=DEV)
    at = torch.arange(P, device=DEV)
    return (e[:, :1] * P + at)[(at >= e[:, 1:2]) & (at < e[:, 2:3])]
