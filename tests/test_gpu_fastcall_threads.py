"""The binding's native calls and Python's other threads (GPU)."""
import subprocess
import threading
import time
import weakref

import pytest
import torch

import sparse_attention_aware_b200 as sa
from sparse_attention_aware_b200 import api
from tests import step_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture
def slow(tmp_path, monkeypatch):
    """The native calls on a library whose functions wait 0.3 s and refuse (so that
    nothing is launched)."""
    import ctypes
    src, so = tmp_path / "slow.c", tmp_path / "slow.so"
    src.write_text("#include <unistd.h>\nlong slow(void) { usleep(300000); return 1; }\n"
                   "unsigned long size(void) { return 256; }\n")
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    real = api._load_fast()
    assert real is not None
    at, size = (ctypes.cast(f, ctypes.c_void_p).value for f in (lib.slow, lib.size))
    monkeypatch.setattr(api, "_fast", real)
    real.init(at, at, at, at, at, size)
    yield real
    api._load_fast()                     # its own functions again


def test_other_threads_run_while_a_call_waits(cuda_dev, slow):
    i32 = dict(dtype=torch.int32, device=cuda_dev)
    g = torch.Generator().manual_seed(1)
    c = sa.PagedCache4(R.random_records(g, 6, 2, 16, 64).to(cuda_dev), torch.arange(6, **i32).view(2, 3),
                       torch.tensor([40, 20], **i32))
    c16 = sa.PagedCache(*(torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16, device=cuda_dev) for _ in range(2)),
                        c.page_table, c.seq_lens)
    x = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=cuda_dev)
    pos, slots = torch.zeros(2, **i32), torch.full((2,), -1, device=cuda_dev)
    sel = sa.TokenSelection(torch.zeros((2, 4, 3), **i32), torch.ones((2, 4), **i32))
    pool = sa.PagePool.full(6, 16, cuda_dev)
    ws = sa.Workspace(cuda_dev)
    raw = torch.cuda.current_stream(cuda_dev).cuda_stream
    ws.at(1 << 16, raw)                  # the workspace has served the stream
    q = x[:, :4].contiguous()
    calls = [lambda: sa.plan_append(c.page_table, c.seq_lens, pos, pool, 4, ws=ws),
             lambda: sa.rope_append(c, x[:, :4], x[:, 4:6], x[:, 6:], pos, slots, ws=ws),
             lambda: sa.rope_append(c16, x[:, :4], x[:, 4:6], x[:, 6:], pos, slots, ws=ws),
             lambda: sa.expand_kv4(c, pos, ws=ws),
             lambda: sa.sparse_decode_attn(c, q, sel, ws=ws)]
    ticks, done = [0], threading.Event()

    def other():
        while not done.is_set():
            ticks[0] += 1
            time.sleep(0.005)

    t = threading.Thread(target=other)
    t.start()
    try:
        for i, call in enumerate(calls):
            before, began = ticks[0], time.monotonic()
            with pytest.raises(sa.SAError):
                call()
            assert time.monotonic() - began >= 0.3, i    # the slow function was called
            # about 60 ticks; with the interpreter held, one at each end
            assert ticks[0] - before >= 10, (i, ticks[0] - before)
    finally:
        done.set()
        t.join()


def test_a_replaced_buffer_outlives_the_native_call_that_uses_it(cuda_dev, slow):
    """Another thread's call outgrows the workspace while a native call on it waits."""
    i32 = dict(dtype=torch.int32, device=cuda_dev)
    table, lens = torch.zeros((2, 3), **i32), torch.zeros(2, **i32)
    pool = sa.PagePool.full(6, 16, cuda_dev)
    ws = sa.Workspace(cuda_dev)
    ws.at(1 << 12, torch.cuda.current_stream(cuda_dev).cuda_stream)
    first, seen = weakref.ref(ws.buf), []

    def grow():
        time.sleep(0.1)                  # the call below waits 0.3 s
        ws.get(1 << 20)
        seen.append((ws.buf is not first(), first() is not None, time.monotonic()))

    t = threading.Thread(target=grow)
    t.start()
    with pytest.raises(sa.SAError):
        sa.plan_append(table, lens, lens, pool, 4, ws=ws)
    done = time.monotonic()
    t.join()
    assert seen[0][:2] == (True, True) and seen[0][2] < done
