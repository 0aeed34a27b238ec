"""Plain 64-bit forms of the serving-step operators, written from their
definitions: page planning, norm + rotary positions, the 4-bit record and
attention over it.  CPU tensors."""
import math

import numpy as np
import torch

BF16_HALF = 2.0 ** -8    # half a step of bf16, relative to the value


# ---------------------------------------------------------------------------
# planning
# ---------------------------------------------------------------------------
def plan(table, lens, new, free, count, page, max_tokens):
    """One token, one page at a time.  Returns the new (table, lens, free,
    count) and (cu, positions, slots, seq_ids)."""
    table, free = table.clone(), free.clone()
    lens = lens.tolist()
    count = int(count)
    for b, a in enumerate(new.tolist()):
        if a < 0:
            for p in range(-(-lens[b] // page)):
                free[count] = table[b, p]
                count += 1
    cu, pos, slots, seqs, out = [0], [], [], [], []
    for b, a in enumerate(new.tolist()):
        n = 0 if a < 0 else lens[b]
        for i in range(max(a, 0)):
            if n % page == 0:
                count -= 1
                table[b, n // page] = free[count]
            pos.append(n)
            slots.append(int(table[b, n // page]) * page + n % page)
            seqs.append(b)
            n += 1
        cu.append(len(pos))
        out.append(n)
    pad = max_tokens - len(pos)
    assert pad >= 0 and count >= 0
    i32 = torch.int32
    return (table, torch.tensor(out, dtype=i32), free, count), \
        (torch.tensor(cu, dtype=i32), torch.tensor(pos + [0] * pad, dtype=i32),
         torch.tensor(slots + [-1] * pad, dtype=torch.int64), torch.tensor(seqs + [-1] * pad, dtype=i32))


# ---------------------------------------------------------------------------
# norm, rotary positions
# ---------------------------------------------------------------------------
def norm_rope(x, weight, eps, pos, inv_freq, interleaved):
    """[T][H][d] -> fp64."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    if inv_freq is None or inv_freq.numel() == 0:
        return x
    n = inv_freq.numel()
    ang = (pos.double()[:, None] * inv_freq.double()[None, :])[:, None, :]
    c, s = torch.cos(ang), torch.sin(ang)
    ia, ib = (torch.arange(0, 2 * n, 2), torch.arange(1, 2 * n, 2)) if interleaved else \
        (torch.arange(n), torch.arange(n, 2 * n))
    y = x.clone()
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


# ---------------------------------------------------------------------------
# the 4-bit record
# ---------------------------------------------------------------------------
def quantize(x):
    """fp64 rows [..., d] -> codes uint8 [..., d], parameters bf16 [..., 2 halves, {scale, zero}]."""
    d = x.shape[-1]
    h = x.reshape(*x.shape[:-1], 2, d // 2)
    lo, hi = h.amin(-1), h.amax(-1)
    scale, zero = ((hi - lo) / 15).float().bfloat16(), lo.float().bfloat16()
    s, z = scale.double()[..., None], zero.double()[..., None]
    t = (h - z) / torch.where(s > 0, s, 1)
    c = torch.where(s > 0, torch.round(t).clamp(0, 15), torch.zeros_like(t))
    bad = ~torch.isfinite(h).all(-1) | ~torch.isfinite(scale.float()) | ~torch.isfinite(zero.float())
    c = torch.where(bad[..., None], torch.zeros_like(c), c)
    nan = torch.full_like(scale, float("nan"))
    par = torch.stack([torch.where(bad, nan, scale), torch.where(bad, nan, zero)], -1)
    return c.reshape(x.shape).to(torch.uint8), par


def records(k, v):
    """fp64 rows [..., d] of keys and values -> records uint8 [..., d + 16]."""
    parts, pars = [], []
    for x in (k, v):
        c, p = quantize(x)
        parts.append(c[..., 0::2] | (c[..., 1::2] << 4))
        pars.append(p.reshape(*p.shape[:-2], 4).contiguous().view(torch.uint8))
    return torch.cat(parts + pars, -1)


def values(rec):
    """Records [..., d + 16] -> fp64 (k, v) [..., d], and the scales [..., 2 (k, v), 2 halves]."""
    d = rec.shape[-1] - 16
    par = rec[..., d:].contiguous().view(torch.bfloat16).double().reshape(*rec.shape[:-1], 2, 2, 2)
    out = []
    for i in range(2):
        b = rec[..., i * d // 2:(i + 1) * d // 2]
        c = torch.stack([b & 15, b >> 4], -1).reshape(*rec.shape[:-1], 2, d // 2).double()
        out.append((par[..., i, :, 1:] + par[..., i, :, :1] * c).reshape(*rec.shape[:-1], d))
    return out[0], out[1], par[..., 0]


def random_records(g, pages, hkv, page, d):
    """A pool of quantised Gaussian rows, keys with a mean per channel."""
    k = torch.randn(pages, hkv, page, d, generator=g).double() + torch.randn(d, generator=g).double()
    v = torch.randn(pages, hkv, page, d, generator=g).double()
    return records(k, v)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def decode(kv, table, q, tokens, scale):
    """tokens(b, h) -> positions.  Returns out [B][H][d], lse [B][H] in fp64, and
    bounds on how far a kernel's may be off (see the terms below)."""
    B, H, d = q.shape
    hkv, P = kv.shape[1], kv.shape[2]
    out = torch.zeros(B, H, d, dtype=torch.float64)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    f32 = q.dtype == torch.float32
    for b in range(B):
        for h in range(H):
            t = torch.as_tensor(tokens(b, h)).long()
            if not t.numel():
                continue
            rec = kv[table[b, t // P].long(), h // (H // hkv), t % P]
            k, v, s = values(rec)
            x = q[b, h].double()
            z = scale * (k @ x)
            lse[b, h] = torch.logsumexp(z, 0)
            w = torch.exp(z - lse[b, h])
            out[b, h] = w @ v
            # score: fp32 sums of terms up to 8 s q and (z + 8 s) q, d of them in 8
            # steps (2^-23 each); an fp32 query keeps 22 of its bits
            big = (8 * s[:, 0].amax(-1) + k.abs().amax(-1) + 15 * s[:, 0].amax(-1)) * x.abs().sum()
            err = float((big * 12 * 2.0 ** -23 + (k.abs() @ x.abs() * 2.0 ** -22 if f32 else 0)).max()) * abs(scale)
            # weights: twice the score's error, ex2 to 2^-22, the product's sums (2^-23 a tile)
            rel = 2 * err + 2.0 ** -20 + t.numel() / 16 * 2.0 ** -23
            half = s[:, 1].amax(0).repeat_interleave(d // 2)          # largest scale of either half
            top = v.abs().amax(0) + 31 * half
            # the rounding of s p (half an fp16 step, 2^-11, times codes up to 8 from the
            # middle), and of the output
            tol_o[b, h] = 2.0 ** -11 * 8 * half + BF16_HALF * out[b, h].abs() + rel * top
            tol_l[b, h] = err + 2.0 ** -20 * (1 + abs(float(lse[b, h])))
    return out, lse, tol_o, tol_l


def check_decode(got, ref, where=""):
    out, lse = got
    o, l, to, tl = ref
    out, lse = out.double().cpu(), lse.double().cpu()
    assert torch.isfinite(out).all(), where
    assert torch.equal(torch.isfinite(lse), torch.isfinite(l)), where
    assert bool(((out - o).abs() <= to).all()), (where, float(((out - o).abs() - to).max()))
    f = torch.isfinite(l)
    assert bool(((lse - l)[f].abs() <= tl[f]).all()), (where, float(((lse - l)[f].abs() - tl[f]).max()))


def entries_of(spans, n, page):
    """[start, end) spans (disjoint, ascending) -> entries {page, lo, hi, tokens before}."""
    out, before = [], 0
    for s, e in spans:
        e = min(e, n)
        while s < e:
            p = s // page
            hi = min(e - p * page, page)
            out.append((p, s - p * page, hi, before))
            before += hi - (s - p * page)
            s = (p + 1) * page
    return out


def pack_entries(lists, most=None):
    most = most or max(1, max(len(x) for x in lists))
    blocks = np.full((len(lists), most, 4), -1, dtype=np.int32)
    for b, x in enumerate(lists):
        if x:
            blocks[b, :len(x)] = x
    return torch.from_numpy(blocks), torch.tensor([len(x) for x in lists], dtype=torch.int32)
