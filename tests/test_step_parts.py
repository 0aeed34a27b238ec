"""The 4-bit decode with its parts in memory of their own: refusals on the host,
before any launch (CPU)."""
import ctypes

import pytest

from sparse_attention_aware_b200 import _lib as L
from sparse_attention_aware_b200 import build as B

OK, INV, WS = 0, 1, 3
AT, PARTS = 0x100000, 0x200000     # fake, aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def _call(lib, batch=2, splits=3, parts=PARTS, parts_bytes=1 << 30, ws=AT, ws_bytes=256):
    c = L.KV4CacheS(0x10000, 0x20000, 0x30000, batch, 2, 128, 16, 8, 16)
    sel = L.SelectionS(L.SEL_TOKENS, 0x60000, 0x70000, 16, None, None, 0)
    return lib.sa_sparse_decode_attn_kv4_parts(ctypes.byref(c), 0x40000, L.DTYPE_BF16, 8, ctypes.byref(sel), 0.1,
                                               splits, 0x50000, None, parts, parts_bytes, ws, ws_bytes, None)


def test_parts_refusals(lib):
    need = lib.sa_kv4_decode_workspace_bytes(
        ctypes.byref(L.KV4CacheS(0x10000, 0x20000, 0x30000, 2, 2, 128, 16, 8, 16)), 8, 3) - 256
    assert need >= 2 * 8 * 3 * (128 + 2) * 4
    assert _call(lib, parts=None) == WS and _call(lib, parts=PARTS + 8) == WS
    assert _call(lib, parts_bytes=need - 1) == WS
    assert _call(lib, ws=None) == WS and _call(lib, ws_bytes=255) == WS and _call(lib, ws=AT + 16) == WS
    assert _call(lib, splits=65) == INV
    # a batch of nothing launches nothing
    assert _call(lib, batch=0, parts_bytes=1 << 20) == OK
