"""Numbers that the serving-step calls cannot take: one refusal, through the native
calls and through Python (GPU)."""
import pytest
import torch

import sparse_attention_aware_b200 as sa
from sparse_attention_aware_b200 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("native", [True, False])
def test_numbers_of_another_type_or_size(cuda_dev, monkeypatch, native):
    if native:
        assert api._load_fast() is not None
    else:
        monkeypatch.setattr(api, "_fast", None)
    i32 = dict(dtype=torch.int32, device=cuda_dev)
    table, lens, ws = torch.zeros((2, 4), **i32), torch.zeros(2, **i32), sa.Workspace(cuda_dev)

    def plan(num_pages=8, page_size=16, max_tokens=4):
        pool = sa.PagePool(torch.arange(8, **i32), torch.tensor([8], **i32), num_pages, page_size)
        return sa.plan_append(table, lens, torch.zeros(2, **i32), pool, max_tokens, ws=ws)

    plan()
    for kw in (dict(max_tokens=4.0), dict(page_size=16.0), dict(num_pages="8"), dict(max_tokens=None)):
        with pytest.raises(TypeError):
            plan(**kw)
    for kw in (dict(num_pages=2 ** 32 + 8), dict(page_size=2 ** 32 + 16), dict(max_tokens=2 ** 32 + 4),
               dict(num_pages=-2 ** 40)):
        with pytest.raises(ValueError, match="32 bits"):
            plan(**kw)
    with pytest.raises(sa.SAError):
        plan(page_size=-16)
    c = sa.PagedCache4.empty(8, 2, 16, 64, table, lens)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=cuda_dev)
    sel = sa.TokenSelection(torch.zeros((2, 4, 3), **i32), torch.zeros((2, 4), **i32))
    sa.sparse_decode_attn(c, q, sel, ws=ws)
    with pytest.raises(TypeError):
        sa.sparse_decode_attn(c, q, sel, num_splits=2.0, ws=ws)
    with pytest.raises(ValueError, match="32 bits"):
        sa.sparse_decode_attn(c, q, sel, num_splits=2 ** 32 + 2, ws=ws)
    assert ws.status()[0] == 0 and plan().slots.tolist() == [-1] * 4
