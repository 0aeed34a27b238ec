"""The scores of the 4-bit decode, bit by bit: a list of one token, whose log-sum-exp
is its score (GPU)."""
import math

import pytest
import torch

import sparse_attention_aware_b200 as sa
from tests import step_ref as R

pytestmark = pytest.mark.gpu


def _rows(dev, g, d, heads, lists, make_query):
    """One-token lists over 4096 rows: the log-sum-exps' distance from the scores in 64
    bits (root of the mean square), and per row what the bounds are made of."""
    hkv, page = 4, 16
    B = 4096 // (hkv * heads)
    k = torch.randn(B, hkv, d, generator=g).double() + torch.randn(d, generator=g).double()
    rec = R.records(k, torch.randn(B, hkv, d, generator=g).double())
    kv = torch.zeros(B, hkv, page, d + 16, dtype=torch.uint8)
    kv[:, :, 0] = rec
    q = make_query(B, hkv, heads, d)
    key = R.values(rec)[0].double()                                     # [B][hkv][d]
    score = torch.einsum("bghd,bgd->bgh", q.double(), key)
    # the two terms of each half: s q.c and z sum(q)
    par = rec[..., d:d + 8].contiguous().view(torch.bfloat16).double().unflatten(-1, (2, 2))
    zero = par[..., 1].repeat_interleave(d // 2, dim=-1)
    a = (q.double() * (key - zero)[:, :, None]).unflatten(-1, (2, d // 2)).sum(-1).abs().sum(-1)
    b = (q.double() * zero[:, :, None]).unflatten(-1, (2, d // 2)).sum(-1).abs().sum(-1)
    i32 = dict(dtype=torch.int32, device=dev)
    c = sa.PagedCache4(kv.to(dev), torch.arange(B, **i32).view(B, 1), torch.ones(B, **i32))
    H = hkv * heads
    if lists:
        sel = sa.TokenSelection(torch.zeros((B, H, 1), **i32), torch.ones((B, H), **i32))
    else:
        sel = sa.BlockSelection(torch.tensor([[[0, 0, 1, 0]]] * B, **i32), torch.ones(B, **i32))
    ws = sa.Workspace(dev)
    _, lse = sa.sparse_decode_attn(c, q.view(B, H, d).to(dev), sel, ws=ws)
    assert ws.status()[0] == 0
    off = float((lse.double().cpu().view(B, hkv, heads) - score / math.sqrt(d)).square().mean().sqrt())
    # at most six fp32 roundings of numbers as large as the terms, three of the score's size
    u = 2.0 ** -24 / math.sqrt(3)
    return off, q.double(), key, par[..., 0].amax(-1)[..., None], 6 * (u * (a + b)) ** 2 + 3 * (u * score) ** 2


@pytest.mark.parametrize("lists", [True, False])
@pytest.mark.parametrize("d,heads", [(64, 4), (128, 1), (128, 4), (128, 8), (128, 12), (64, 16)])
def test_scores_of_fp32_queries(cuda_dev, d, heads, lists):
    """What the score of an fp32 query may be off by, from the kernel's arithmetic.

    The query is scaled by 2^n, its largest element to [2^10, 2^11), and is the nearest
    whole numbers, exact, and rests of up to 1/2 in fp16: evenly spread rests are off by
    0.436 * 2^-13 (root of the mean square: 2^-13 / sqrt 3 for those above 1/4, half of it
    for each halving below).  At most six fp32 roundings, of 2^-24 / sqrt 3 each, are of
    numbers as large as the halves' terms s q.c and z sum(q) together, and three of the
    score's size.  Errors of 4096 rows are taken together, and twice the sum is allowed."""
    g = torch.Generator().manual_seed(100 * d + heads)
    off, q, key, _, rounded = _rows(cuda_dev, g, d, heads, lists, lambda *s: torch.randn(*s, generator=g))
    unit = 2.0 ** (torch.floor(torch.log2(q.abs().amax(-1))) - 10)
    rest = 0.436 * 2.0 ** -13 * unit * key.norm(dim=-1)[..., None]
    allowed = 2 / math.sqrt(d) * float((rest ** 2 + rounded).mean().sqrt())
    assert off <= allowed, (off, allowed)


@pytest.mark.parametrize("lists", [True, False])
@pytest.mark.parametrize("kind", ["even", "spread", "one large"])
@pytest.mark.parametrize("d,heads", [(64, 4), (128, 1), (128, 4), (128, 8), (64, 12), (128, 16)])
def test_scores_of_bf16_queries(cuda_dev, d, heads, kind, lists):
    """A bf16 query of Gaussian elements, of elements of very different sizes, and of ones
    of like sizes with a channel that is 2^9 times as large.

    The query is exact; of each product of an element and a code, what lies below 2^-18
    of the largest element is dropped, which only elements below 2^-10 of it have: a
    unit of 2^-18 of it times the scale at most for each of those, and nothing that
    evens out.  The fp32 roundings are as above."""
    g = torch.Generator().manual_seed(200 * d + 10 * heads + len(kind))

    def query(*shape):
        x = torch.randn(*shape, generator=g)
        if kind == "spread":
            x = x * torch.exp(2 * torch.randn(*shape, generator=g))
        if kind == "one large":
            x = torch.sign(x) * (0.5 + 0.5 * torch.rand(*shape, generator=g).clamp(max=0.99))
            x.scatter_(-1, torch.randint(0, d, (*shape[:-1], 1), generator=g), 256.0)
        return x.bfloat16()

    off, q, _, step, rounded = _rows(cuda_dev, g, d, heads, lists, query)
    top = q.abs().amax(-1)
    few = (q.abs() < 2.0 ** -10 * top[..., None]).sum(-1)
    dropped = few * 2.0 ** -18 * top * step
    allowed = 2 / math.sqrt(d) * float((rounded + dropped ** 2).mean().sqrt())
    assert off <= allowed, (off, allowed)
