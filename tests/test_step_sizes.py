"""Sizes next to what 32 bits count: the serving-step calls refuse them on the host,
before any launch (CPU)."""
import ctypes

import pytest

from sparse_attention_aware_b200 import _lib as L
from sparse_attention_aware_b200 import build as B

INV, UNS = 1, 2
AT, ROOM = 0x100000, 1 << 40     # fake, aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


@pytest.mark.parametrize("field", ["max_tokens", "num_free"])
@pytest.mark.parametrize("size", [2 ** 30 + 1, 2 ** 31 - 200, 2 ** 31 - 1])
def test_plan_sizes(lib, field, size):
    f = dict(page_table=0x1000, seq_lens=0x2000, new_lens=0x3000, free_pages=0x4000, free_count=0x5000,
             seq_lens_out=0x6000, free_count_out=0x7000, cu_tokens=0x8000, positions=0x9000, slots=0xa000,
             seq_ids=0xb000, batch=3, page_size=16, max_pages_per_seq=8, num_pages=24, num_free=24, max_tokens=10)
    f[field] = size
    a = L.PlanArgsS(**f)
    assert lib.sa_plan_append(ctypes.byref(a), AT, ROOM, None) == UNS
    f[field] = 2 ** 30                  # taken: refused for another field alone
    f["cu_tokens"] = None
    assert lib.sa_plan_append(ctypes.byref(L.PlanArgsS(**f)), AT, ROOM, None) == INV


@pytest.mark.parametrize("size", [2 ** 30 + 1, 2 ** 31 - 300, 2 ** 31 - 1])
@pytest.mark.parametrize("splits", [0, 1, 64])
def test_list_sizes(lib, size, splits):
    c = L.KV4CacheS(0x10000, 0x20000, 0x30000, 2, 2, 128, 16, 8, 16)
    for sel in (L.SelectionS(L.SEL_TOKENS, 0x60000, 0x70000, size, None, None, 0),
                L.SelectionS(L.SEL_BLOCKS, None, None, 0, 0x60000, 0x70000, size)):
        assert lib.sa_sparse_decode_attn_kv4(ctypes.byref(c), 0x40000, L.DTYPE_BF16, 8, ctypes.byref(sel), 0.1, splits,
                                             0x50000, None, AT, ROOM, None) == UNS
