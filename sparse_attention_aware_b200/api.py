"""Python binding of libsa: the four entry points with the C ABI's names.

Argument marshalling only: tensors are passed to the C library as raw device
pointers on torch's current stream, outputs and workspaces are allocated with
torch when the caller does not pass them.  Every step of the computation runs
in libsa's CUDA kernels; if the library is missing, ``_lib.load`` raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import inspect
import math
import operator
import threading
import warnings
from typing import Optional, Sequence

import torch

from . import _lib as L
from .cache import PagedCache4, PagePool


class SAError(RuntimeError):
    def __init__(self, status: int, where: str, detail=None):
        self.status = status
        self.detail = detail
        msg = "%s: %s" % (where, L.load().sa_status_string(status).decode())
        if detail is not None:
            msg += " (check %d, value %d)" % (detail[1], detail[2])
        super().__init__(msg)


def _check(status: int, where: str):
    if status != L.SA_OK:
        raise SAError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _load_fast():
    """The native short way of the calls below (csrc/fastcall.cpp), set up with
    libsa's entry points; None, with a warning, where it has not been built for
    this torch and Python (it uses torch's own C++ classes)."""
    from . import build
    try:
        if not build.fastcall_fits():
            raise ImportError("%s is missing, or compiled against another torch or Python" % build.FAST)
        from . import _fastcall
    except ImportError as e:
        warnings.warn("calls take 8 to 20 us longer without the binding's native calls (%s); "
                      "python -m sparse_attention_aware_b200.build makes them" % e, RuntimeWarning)
        return None
    lib = L.load()
    _fastcall.init(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in
                     ("sa_plan_append", "sa_rope_append", "sa_rope_append_kv4", "sa_expand_kv4",
                      "sa_sparse_decode_attn_kv4", "sa_kv4_decode_workspace_bytes")))
    return _fastcall


_fast = False   # False: not looked for yet


def _short(ws: Optional[Workspace], device, stream):
    """(native calls, workspace address, bytes, stream handle, what keeps the
    buffer) if a call may go the short way: it is on torch's current stream, with
    a workspace that has served that stream before."""
    global _fast
    if _fast is False:
        _fast = _load_fast()
    if _fast is None or stream is not None or device.type != "cuda":
        return None
    raw = _raw_stream(device.index)
    if ws is None:
        ws = _default_ws_at.get((device.index, raw))
        if ws is None:
            return None
    at = ws._raw.get(raw) if ws._index == device.index else None   # (handles of two devices' streams may be alike)
    return None if at is None else (_fast, at[0], at[1], raw, at)


def _raw_stream(index: int) -> int:
    """Handle of torch's current stream on device ``index``."""
    return _current_raw(index) if _current_raw is not None else torch.cuda.current_stream(index).cuda_stream


# torch's own accessor of the bare handle (current_stream builds an object: 8 us a call)
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on_call_stream(fn):
    """When an entry point is given ``stream=``, the tensors it makes itself
    (contiguous copies of inputs, threshold tensors, default outputs, a
    growing workspace) are made on that stream, so that they are ordered
    before the kernels that read them and the caching allocator does not hand
    their memory out again while those kernels run.  Without ``stream=`` the
    call runs on torch's current stream as before."""
    @functools.wraps(fn)
    def call(*args, **kw):
        s = kw.get("stream")
        if s is None:
            return fn(*args, **kw)
        with torch.cuda.stream(s):
            return fn(*args, **kw)
    return call


def kv_struct(cache, device=None) -> L.KVCacheS:
    """``cache``: any object with k, v, page_table, seq_lens tensors on the GPU
    (k/v bf16 [num_pages][Hkv][P][d], page_table int32 [B][max_pages],
    seq_lens int32 [B]).  ``device``: when given, every cache tensor must be on
    it (the device of the call's queries).  Raises ValueError otherwise."""
    if isinstance(cache, PagedCache4):
        raise TypeError("this call reads bf16 pages: expand_kv4 gives those of a 4-bit cache")
    k, v = cache.k, cache.v
    pt, sl = cache.page_table, cache.seq_lens
    if k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise ValueError("KV cache: k and v must be bf16, got %s / %s" % (k.dtype, v.dtype))
    if k.dim() != 4 or k.shape != v.shape or not k.is_contiguous() or not v.is_contiguous():
        raise ValueError("KV cache: k and v must be contiguous [num_pages][Hkv][P][d] tensors of one shape")
    if pt.dtype != torch.int32 or pt.dim() != 2 or not pt.is_contiguous():
        raise ValueError("KV cache: page_table must be a contiguous int32 [B][max_pages] tensor")
    if sl.dtype != torch.int32 or tuple(sl.shape) != (pt.shape[0],) or not sl.is_contiguous():
        raise ValueError("KV cache: seq_lens must be a contiguous int32 [B] tensor, B = %d" % pt.shape[0])
    devs = {t.device for t in (k, v, pt, sl)}
    if device is not None:
        devs.add(torch.device(device))
    if len(devs) != 1:
        raise ValueError("KV cache: k, v, page_table, seq_lens and the queries must be on one device, got %s"
                         % sorted(str(d) for d in devs))
    return L.KVCacheS(k.data_ptr(), v.data_ptr(), pt.data_ptr(), sl.data_ptr(), pt.shape[0], k.shape[1],
                      k.shape[3], k.shape[2], pt.shape[1], k.shape[0])


def kv4_struct(cache: PagedCache4, device=None) -> L.KV4CacheS:
    """``kv_struct`` for a 4-bit cache."""
    kv, pt, sl = cache.kv, cache.page_table, cache.seq_lens
    n, h, p, r = kv.shape if kv.dim() == 4 else (0, 0, 0, 0)
    if kv.dtype is not torch.uint8 or r <= 16 or not kv.is_contiguous():
        raise ValueError("4-bit KV cache: kv must be a contiguous uint8 [num_pages][Hkv][P][d + 16] tensor")
    B, mp = pt.shape if pt.dim() == 2 else (0, 0)
    if pt.dtype is not torch.int32 or pt.dim() != 2 or not pt.is_contiguous():
        raise ValueError("4-bit KV cache: page_table must be a contiguous int32 [B][max_pages] tensor")
    if sl.dtype is not torch.int32 or sl.shape != (B,) or not sl.is_contiguous():
        raise ValueError("4-bit KV cache: seq_lens must be a contiguous int32 [B] tensor, B = %d" % pt.shape[0])
    dev = kv.device
    if pt.device != dev or sl.device != dev or (device is not None and dev != device):
        raise ValueError("4-bit KV cache: kv, page_table, seq_lens and the queries must be on one device, got %s"
                         % sorted({str(t.device) for t in (kv, pt, sl)} | {str(device)}))
    return L.KV4CacheS(kv.data_ptr(), pt.data_ptr(), sl.data_ptr(), B, h, r - 16, p, mp, n)


def _geometry(cache, device=None) -> L.KVCacheS:
    """``kv_struct``, where a 4-bit cache is its lengths and page geometry (all
    that the span selection reads)."""
    if not isinstance(cache, PagedCache4):
        return kv_struct(cache, device)
    c = kv4_struct(cache, device)
    return L.KVCacheS(None, None, c.page_table, c.seq_lens, c.batch, c.num_kv_heads, c.head_dim, c.page_size,
                      c.max_pages_per_seq, c.num_pages)


def _capturing() -> bool:
    """Whether torch's current stream is being captured into a graph."""
    return torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing()


def _aligned(buf: torch.Tensor) -> int:
    """Where a workspace begins in its buffer."""
    return (buf.data_ptr() + 255) // 256 * 256


class Workspace:
    """A reusable, zero-initialised device workspace (grows on demand).

    A workspace belongs to one stream at a time: calls that share it must be
    ordered on the GPU (same stream, or events between streams), since every
    call rewrites its status header and scratch.  When it grows, the old
    buffer is released with record_stream() for every stream it was handed
    to, so the caching allocator does not reuse that memory while a kernel
    launched on one of those streams may still read it.  A buffer that a
    captured call was handed is kept instead: every replay of that graph writes
    to it again, and ``status`` reads it too.  A workspace that is captured must
    outlive its graphs; one that is made by a captured call is cleared by every
    replay of that call's graph.  Graphs that share one are replayed one after the
    other, unless their calls use its status word alone (``plan_append``,
    ``rope_append``, ``expand_kv4``).

    What gives a call its address keeps the buffer as well, and the call holds it
    until it has launched: another thread's call on the same stream may replace
    the buffer in between, but its memory is let go, behind the launch, by the
    last call that holds it."""

    def __init__(self, device=None):
        self.device = device
        self.buf: Optional[torch.Tensor] = None
        self._index = None   # of buf's device
        self._streams = []
        self._raw = {}   # stream handles in _streams -> (aligned address of buf, bytes from there on, buf)
        self._grow = threading.Lock()
        self._in_graph = False   # buf was handed to a captured call
        self._kept = []          # outgrown buffers that were

    def _zeros(self, n: int) -> torch.Tensor:
        return torch.zeros(n, dtype=torch.uint8, device=self.device or "cuda")

    def at(self, nbytes: int, raw: int, stream=None):
        """(address, bytes, what keeps the buffer) for a call on the stream of handle
        ``raw``, without asking torch for its stream object when the buffer has
        served it before."""
        got = self._raw.get(raw)
        if got is not None and got[1] >= nbytes:
            if _capturing():
                self._captured(got[2])
            return got
        buf = self.get(nbytes + 256, stream)
        at = _aligned(buf)
        got = at, buf.numel() - (at - buf.data_ptr()), buf
        with self._grow:
            if self.buf is buf:
                self._raw[raw] = got
        return got

    def get(self, nbytes: int, stream=None) -> torch.Tensor:
        buf = self.buf
        if buf is None or buf.numel() < nbytes:
            with self._grow:
                buf = self.buf
                if buf is None or buf.numel() < nbytes:
                    buf = self._zeros(max(nbytes, 256) + 256)
                    if self.buf is not None and self._in_graph:
                        self._kept.append(self.buf)
                    elif self.buf is not None:
                        for s in self._streams:
                            self.buf.record_stream(s)
                    self._streams = []
                    self._raw = {}
                    self._in_graph = False
                    self._index = buf.device.index
                    self.buf = buf
        if _capturing():
            self._captured(buf)
        if buf.device.type == "cuda":
            s = stream if stream is not None else torch.cuda.current_stream(buf.device)
            if all(s != x for x in self._streams):
                self._streams.append(s)
                if self.buf is not buf:   # replaced since, and released for the streams that were known
                    buf.record_stream(s)
        return buf

    def _captured(self, buf: torch.Tensor) -> None:
        """``buf`` is handed to a captured call."""
        with self._grow:
            if self.buf is buf:
                self._in_graph = True
            elif all(buf is not x for x in self._kept):
                self._kept.append(buf)

    def aligned(self, nbytes: int, stream=None):
        buf = self.get(nbytes, stream)
        at = _aligned(buf)
        ptr = ctypes.c_void_p(at)
        ptr.held = buf
        return ptr, buf.numel() - (at - buf.data_ptr())

    def status(self, stream=None):
        """Synchronise and return (status, detail) recorded by kernels (then cleared)."""
        found = 0, (0, 0, 0)
        for buf in self._kept + ([] if self.buf is None else [self.buf]):
            det = (L.c_i32 * 3)()
            st = L.load().sa_read_device_status(ctypes.c_void_p(_aligned(buf)), _stream(stream), det)
            if st != 0 and found[0] == 0:
                found = st, tuple(det)
        return found

    def raise_on_fault(self, where="device", stream=None):
        st, det = self.status(stream)
        if st != 0:
            raise SAError(st, where, det)


def _zeros_outside_graph(n: int, device) -> torch.Tensor:
    """Zeroed device memory that belongs to no graph, while torch's current stream
    is being captured: made, cleared and waited for on a stream that is not.
    (Memory of a graph's pool would be cleared by its replays, and not before
    the first.)"""
    lib = ctypes.CDLL("libcuda.so.1")
    mode = ctypes.c_int(2)   # relaxed: other streams may be waited for
    lib.cuThreadExchangeStreamCaptureMode(ctypes.byref(mode))
    try:
        while True:   # (torch hands its streams out in turn, the captured one too)
            side = torch.cuda.Stream(device)
            with torch.cuda.stream(side):
                if not torch.cuda.is_current_stream_capturing():
                    buf = torch.zeros(n, dtype=torch.uint8, device=device)
                    break
        side.synchronize()
    finally:
        lib.cuThreadExchangeStreamCaptureMode(ctypes.byref(mode))
    return buf


class _DefaultWorkspace(Workspace):
    """The workspace of a stream's calls that were given none.  It lives as long as
    the process, and so it may be made by a captured call."""

    def _zeros(self, n: int) -> torch.Tensor:
        return _zeros_outside_graph(n, self.device) if _capturing() else super()._zeros(n)


def device_status(device=None):
    """(status, detail) of the calls on ``device`` (the current one) that were
    given no workspace: the first record found in their streams' workspaces, which
    are then cleared.  Waits for the device.  Replays of such calls that were
    captured record here too."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    found = 0, (0, 0, 0)
    with torch.cuda.device(dev):
        torch.cuda.synchronize()
        for ws in list(_default_ws.values()):
            if ws.buf is not None and ws.buf.device.type == "cuda" and ws.buf.device.index == torch.cuda.current_device():
                got = ws.status()
                found = got if found[0] == 0 else found
    return found


_default_ws = {}
_default_ws_at = {}   # (device index, stream handle) -> the same workspaces


def _scratch(ws: Optional[Workspace], dev: torch.device, stream, nbytes: int):
    """The workspace of a call (the caller's, else the default one of its device
    and stream) and the stream's handle: (address, bytes, handle, what keeps the
    buffer).  Raises ValueError for a workspace or a stream of another device."""
    if stream is not None and stream.device != dev:
        raise ValueError("the call's tensors are on %s, its stream is on %s" % (dev, stream.device))
    if ws is not None and (ws.buf is not None or ws.device is not None):
        on = ws.buf.device if ws.buf is not None else torch.device(ws.device)
        if on.type != dev.type or on.index not in (None, dev.index):
            raise ValueError("the call's tensors are on %s, its workspace is on %s" % (dev, on))
    raw = _raw_stream(dev.index) if stream is None else stream.cuda_stream
    if ws is None:
        ws = _default_ws_at.get((dev.index, raw))
        if ws is None:
            ws = _default_ws_at[(dev.index, raw)] = _ws(None, dev, stream)
    at = ws.at(nbytes, raw, stream)
    return at[0], at[1], raw, at


def _ws(ws: Optional[Workspace], device, stream=None) -> Workspace:
    """The caller's workspace, else a default one per (device, stream), so
    that calls on different streams never share scratch."""
    if ws is not None:
        return ws
    dev = torch.device(device)
    if stream is not None:
        sid = int(stream.cuda_stream)
    elif dev.type == "cuda":
        sid = int(torch.cuda.current_stream(dev).cuda_stream)
    else:
        sid = 0
    key = (str(dev), sid)
    if key not in _default_ws:
        _default_ws[key] = _DefaultWorkspace(device)
    return _default_ws[key]


def workspace_bytes(op: int, cache, num_q_heads=0, k=0, num_splits=0, num_tokens=0,
                    block_args: Optional[L.BlockSelectArgsS] = None) -> int:
    kv = _geometry(cache)
    q = L.WsQueryS(num_q_heads, k, num_splits, num_tokens,
                   ctypes.pointer(block_args) if block_args is not None else None)
    n = L.load().sa_workspace_bytes(op, ctypes.byref(kv), ctypes.byref(q))
    if n == 0:
        raise SAError(1, "sa_workspace_bytes")
    return n


def _need(t: torch.Tensor, shape, dtype, device, what: str) -> None:
    """A caller-provided output (or index) tensor must have exactly the layout
    the library writes: shape, dtype, contiguity and device."""
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or t.device != device:
        raise ValueError("%s: need a contiguous %s tensor of shape %s on %s, got %s %s on %s"
                         % (what, dtype, tuple(shape), device, t.dtype, tuple(t.shape), t.device))


def _int32(x, what: str) -> None:
    """A size that the library takes as 32 bits (ctypes would cut it)."""
    if not -2 ** 31 <= operator.index(x) < 2 ** 31:
        raise ValueError("%s: %d needs more than 32 bits" % (what, x))


def _bf16_q(q: torch.Tensor, what: str) -> torch.Tensor:
    if q.dtype != torch.bfloat16:
        raise TypeError("%s: q must be bf16, got %s" % (what, q.dtype))
    return q.contiguous()


def _qdtype(q: torch.Tensor) -> int:
    if q.dtype == torch.float32:
        return L.DTYPE_F32
    if q.dtype == torch.bfloat16:
        return L.DTYPE_BF16
    raise TypeError("q must be fp32 or bf16")


def _on_call_device(fn):
    """``_on_call_stream``, and the call's kernels go to the device of the
    call's first tensor also where that is not the current one."""
    first = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, **kw):
        s = kw.get("stream")
        if s is not None:
            with torch.cuda.stream(s):
                return fn(*args, **kw)
        x = args[0] if args else kw[first]
        dev = x.device if isinstance(x, torch.Tensor) else x.kv.device if isinstance(x, PagedCache4) else x.k.device
        if dev.type != "cuda" or dev.index == torch.cuda.current_device():
            return fn(*args, **kw)
        with torch.cuda.device(dev):
            return fn(*args, **kw)
    return call


# --------------------------------------------------------------------------
# selections
# --------------------------------------------------------------------------
@dataclasses.dataclass
class TokenSelection:
    idx: torch.Tensor     # int32 [B][Hq][k_cap]
    count: torch.Tensor   # int32 [B][Hq]

    def struct(self) -> L.SelectionS:
        return L.SelectionS(L.SEL_TOKENS, self.idx.data_ptr(), self.count.data_ptr(), self.idx.shape[-1],
                            None, None, 0)


@dataclasses.dataclass
class BlockSelection:
    blocks: torch.Tensor        # int32 [B][max_blocks][4]
    block_counts: torch.Tensor  # int32 [B]

    def struct(self) -> L.SelectionS:
        return L.SelectionS(L.SEL_BLOCKS, None, None, 0, self.blocks.data_ptr(),
                            self.block_counts.data_ptr(), self.blocks.shape[1])


@dataclasses.dataclass
class BlockCSR:
    row_ptr: torch.Tensor   # int32 [Hq*nQB + 1]
    cols: torch.Tensor      # int32 [nnz_capacity]
    tau: torch.Tensor       # fp32 [2][Hq] thresholds applied
    num_q_heads: int
    num_q_blocks: int


def _check_selection(sel, B: int, Hq: int, device) -> None:
    """The selection tensors a decode reads must have the layout the kernels
    index: token lists idx int32 [B][Hq][k_cap] and count int32 [B][Hq];
    block lists blocks int32 [B][max_blocks][4] and block_counts int32 [B];
    contiguous, on the queries' device.  Raises ValueError otherwise."""
    if isinstance(sel, TokenSelection):
        if sel.idx.dim() != 3:
            raise ValueError("TokenSelection.idx must be int32 [B][Hq][k_cap], got shape %s" % (tuple(sel.idx.shape),))
        _need(sel.idx, (B, Hq, sel.idx.shape[-1]), torch.int32, device, "TokenSelection.idx")
        _need(sel.count, (B, Hq), torch.int32, device, "TokenSelection.count")
    elif isinstance(sel, BlockSelection):
        if sel.blocks.dim() != 3:
            raise ValueError("BlockSelection.blocks must be int32 [B][max_blocks][4], got shape %s"
                             % (tuple(sel.blocks.shape),))
        _need(sel.blocks, (B, sel.blocks.shape[1], 4), torch.int32, device, "BlockSelection.blocks")
        _need(sel.block_counts, (B,), torch.int32, device, "BlockSelection.block_counts")
    else:
        raise TypeError("selection must be a TokenSelection or a BlockSelection, got %s" % type(sel).__name__)


# --------------------------------------------------------------------------
# entry points
# --------------------------------------------------------------------------
@_on_call_stream
def select_topk(cache, q: torch.Tensor, k: int, idx: Optional[torch.Tensor] = None,
                count: Optional[torch.Tensor] = None, ws: Optional[Workspace] = None,
                stream=None) -> TokenSelection:
    """Anchor-layer exact top-k per query head (``sa_select_topk``)."""
    B, Hq, d = q.shape
    dev = q.device
    if idx is None:
        idx = torch.empty((B, Hq, k), dtype=torch.int32, device=dev)
    _need(idx, (B, Hq, k), torch.int32, dev, "select_topk idx")
    if count is None:
        count = torch.empty((B, Hq), dtype=torch.int32, device=dev)
    _need(count, (B, Hq), torch.int32, dev, "select_topk count")
    kv = kv_struct(cache, dev)
    w = _ws(ws, dev, stream)
    wp, wn = w.aligned(workspace_bytes(L.OP_SELECT_TOPK, cache, num_q_heads=Hq, k=k), stream)
    _check(L.load().sa_select_topk(ctypes.byref(kv), _ptr(q.contiguous()), _qdtype(q), Hq, k, _ptr(idx),
                                   _ptr(count), wp, wn, _stream(stream)), "sa_select_topk")
    return TokenSelection(idx, count)


@_on_call_stream
def sparse_decode_attn(cache, q: torch.Tensor, sel, scale: Optional[float] = None,
                       num_splits: Optional[int] = None,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       want_lse: bool = True, ws: Optional[Workspace] = None, stream=None):
    """Split-KV sparse decode + combine (``sa_sparse_decode_attn``, or
    ``sa_sparse_decode_attn_kv4`` over a PagedCache4).  ``num_splits`` parts a
    list, 1 by default; over a PagedCache4 0, the default there, lets the
    library choose by the selection's capacity (for masks far below the context
    give ``select_blocks_spans`` the ``max_blocks`` they need).  Captured into a graph without ``ws``, a call over a
    PagedCache4 keeps its parts in that graph's memory, so that graphs may be
    replayed side by side; what its replays record, ``device_status`` reads.
    Returns (out bf16, lse fp32)."""
    if isinstance(cache, PagedCache4):
        return _decode_kv4(cache, q, sel, scale, 0 if num_splits is None else num_splits, out, lse, want_lse, ws, stream)
    if num_splits is None:
        num_splits = 1
    B, Hq, d = q.shape
    dev = q.device
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.bfloat16, device=dev)
    _need(out, (B, Hq, d), torch.bfloat16, dev, "sparse_decode_attn out")
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    if lse is not None:
        _need(lse, (B, Hq), torch.float32, dev, "sparse_decode_attn lse")
    kv = kv_struct(cache, dev)
    _check_selection(sel, B, Hq, dev)
    s = sel.struct()
    w = _ws(ws, dev, stream)
    wp, wn = w.aligned(workspace_bytes(L.OP_DECODE, cache, num_q_heads=Hq, num_splits=num_splits), stream)
    _check(L.load().sa_sparse_decode_attn(ctypes.byref(kv), _ptr(q.contiguous()), _qdtype(q), Hq,
                                          ctypes.byref(s), scale, num_splits, _ptr(out), _ptr(lse), wp, wn,
                                          _stream(stream)), "sa_sparse_decode_attn")
    return out, lse


def _decode_kv4(cache: PagedCache4, q, sel, scale, num_splits, out, lse, want_lse, ws, stream):
    if out is None and lse is None:
        way = _short(ws, q.device, stream)
        if way is not None:
            tok = isinstance(sel, TokenSelection)
            if tok or isinstance(sel, BlockSelection):
                fast, wp, wn, raw, _ = way
                got = fast.decode(cache.kv, cache.page_table, cache.seq_lens, q, sel.idx if tok else sel.blocks,
                                  sel.count if tok else sel.block_counts, L.SEL_TOKENS if tok else L.SEL_BLOCKS, scale,
                                  num_splits, want_lse, wp, wn, raw)
                if got is not None:
                    if isinstance(got, int):
                        _check(got, "sa_sparse_decode_attn_kv4")
                    return got
    return _decode_kv4_checked(cache, q, sel, scale, num_splits, out, lse, want_lse, ws, stream)


@_on_call_device
def _decode_kv4_checked(cache: PagedCache4, q, sel, scale, num_splits, out, lse, want_lse, ws, stream):
    B, Hq, d = q.shape
    dev = q.device
    _int32(num_splits, "sparse_decode_attn num_splits")
    kv = kv4_struct(cache, dev)
    if (B, d) != (kv.batch, kv.head_dim):
        raise ValueError("sparse_decode_attn: q is [%d][%d][%d], the 4-bit cache has batch %d and head_dim %d"
                         % (B, Hq, d, kv.batch, kv.head_dim))
    q = q.contiguous()
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.bfloat16, device=dev)
    else:
        _need(out, (B, Hq, d), torch.bfloat16, dev, "sparse_decode_attn out")
    if lse is not None:
        _need(lse, (B, Hq), torch.float32, dev, "sparse_decode_attn lse")
    elif want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    _check_selection(sel, B, Hq, dev)
    s = sel.struct()
    lib = L.load()
    need = lib.sa_kv4_decode_workspace_bytes(ctypes.byref(kv), Hq, num_splits)
    call = (ctypes.byref(kv), q.data_ptr(), _qdtype(q), Hq, ctypes.byref(s),
            1.0 / math.sqrt(d) if scale is None else scale, num_splits, out.data_ptr(),
            None if lse is None else lse.data_ptr())
    if ws is None and _capturing():
        # graphs may be replayed side by side: each call keeps its parts in its graph's own memory
        wp, wn, raw, _ = _scratch(None, dev, stream, 256)
        parts = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        _check(lib.sa_sparse_decode_attn_kv4_parts(*call, parts.data_ptr(), parts.numel(), wp, wn, raw),
               "sa_sparse_decode_attn_kv4_parts")
        return out, lse
    wp, wn, raw, _ = _scratch(ws, dev, stream, need)
    _check(lib.sa_sparse_decode_attn_kv4(*call, wp, wn, raw), "sa_sparse_decode_attn_kv4")
    return out, lse


# --------------------------------------------------------------------------
# a step's pages, keys and values
# --------------------------------------------------------------------------
@dataclasses.dataclass
class AppendPlan:
    """Where a step's tokens go (``plan_append``)."""
    cu_tokens: torch.Tensor   # int32 [B + 1] first token of each sequence, and their number
    positions: torch.Tensor   # int32 [max_tokens] position in the sequence (0 past the last token)
    slots: torch.Tensor       # int64 [max_tokens] page * P + offset (-1 past the last token)
    seq_ids: torch.Tensor     # int32 [max_tokens] sequence (-1 past the last token)

    @staticmethod
    def empty(batch: int, max_tokens: int, device) -> "AppendPlan":
        return AppendPlan(torch.empty(batch + 1, dtype=torch.int32, device=device),
                          torch.empty(max_tokens, dtype=torch.int32, device=device),
                          torch.empty(max_tokens, dtype=torch.int64, device=device),
                          torch.empty(max_tokens, dtype=torch.int32, device=device))


def plan_append(page_table: torch.Tensor, seq_lens: torch.Tensor, new_lens: torch.Tensor, pool: PagePool,
                max_tokens: int, seq_lens_out: Optional[torch.Tensor] = None,
                free_count_out: Optional[torch.Tensor] = None, plan: Optional[AppendPlan] = None,
                ws: Optional[Workspace] = None, stream=None) -> AppendPlan:
    """Pages, positions and slots of a step from the sequences' lengths
    (``sa_plan_append``): ``new_lens[b]`` tokens are appended to sequence b (-1:
    it has ended).  The page table and the pool's stack are updated in place,
    and so are ``seq_lens`` and ``pool.free_count`` unless ``seq_lens_out`` /
    ``free_count_out`` take the new values.  A step that does not fit changes
    nothing, gives every token slot -1 and is recorded in the workspace."""
    if plan is None:
        way = _short(ws, page_table.device, stream)
        if way is not None:
            fast, wp, wn, raw, _ = way
            got = fast.plan(page_table, seq_lens, new_lens, pool.free_pages, pool.free_count, pool.num_pages,
                            pool.page_size, max_tokens, seq_lens_out, free_count_out, wp, wn, raw)
            if got is not None:
                if isinstance(got, int):
                    _check(got, "sa_plan_append")
                return AppendPlan(*got)
    return _plan_append(page_table, seq_lens, new_lens, pool, max_tokens, seq_lens_out, free_count_out, plan, ws,
                        stream=stream)


@_on_call_device
def _plan_append(page_table, seq_lens, new_lens, pool, max_tokens, seq_lens_out, free_count_out, plan, ws,
                 stream=None) -> AppendPlan:
    dev = page_table.device
    if page_table.dim() != 2:
        raise ValueError("plan_append: page_table must be int32 [B][max_pages]")
    B, mp = page_table.shape
    _need(page_table, (B, mp), torch.int32, dev, "plan_append page_table")
    _need(seq_lens, (B,), torch.int32, dev, "plan_append seq_lens")
    _need(new_lens, (B,), torch.int32, dev, "plan_append new_lens")
    _need(pool.free_pages, (pool.free_pages.numel(),), torch.int32, dev, "plan_append pool.free_pages")
    _need(pool.free_count, (1,), torch.int32, dev, "plan_append pool.free_count")
    _int32(pool.num_pages, "plan_append pool.num_pages")
    _int32(pool.page_size, "plan_append pool.page_size")
    _int32(max_tokens, "plan_append max_tokens")
    if seq_lens_out is None:
        seq_lens_out = seq_lens
    else:
        _need(seq_lens_out, (B,), torch.int32, dev, "plan_append seq_lens_out")
    if free_count_out is None:
        free_count_out = pool.free_count
    else:
        _need(free_count_out, (1,), torch.int32, dev, "plan_append free_count_out")
    if plan is None:
        plan = AppendPlan.empty(B, max_tokens, dev)
    else:
        _need(plan.cu_tokens, (B + 1,), torch.int32, dev, "plan_append plan.cu_tokens")
        _need(plan.positions, (max_tokens,), torch.int32, dev, "plan_append plan.positions")
        _need(plan.slots, (max_tokens,), torch.int64, dev, "plan_append plan.slots")
        _need(plan.seq_ids, (max_tokens,), torch.int32, dev, "plan_append plan.seq_ids")
    a = L.PlanArgsS(page_table.data_ptr(), seq_lens.data_ptr(), new_lens.data_ptr(), pool.free_pages.data_ptr(),
                    pool.free_count.data_ptr(), seq_lens_out.data_ptr(), free_count_out.data_ptr(),
                    plan.cu_tokens.data_ptr(), plan.positions.data_ptr(), plan.slots.data_ptr(),
                    plan.seq_ids.data_ptr(), B, pool.page_size, mp, pool.num_pages, pool.free_pages.numel(),
                    max_tokens)
    wp, wn, raw, _ = _scratch(ws, dev, stream, 256)
    _check(L.load().sa_plan_append(ctypes.byref(a), wp, wn, raw), "sa_plan_append")
    return plan


def _rows(x: torch.Tensor, what: str, shape, device):
    """``x`` as the library reads it -- bf16 [T][H][d] with heads contiguous and
    tokens a multiple of 8 elements apart, 16-byte aligned (parts of a packed
    projection are taken as they are; other layouts are copied) -- and the
    elements between its tokens."""
    if x.dtype is not torch.bfloat16:
        raise TypeError("rope_append: %s must be bf16, got %s" % (what, x.dtype))
    if x.shape != shape or x.device != device:
        raise ValueError("rope_append: %s must be %s on %s, got %s on %s"
                         % (what, shape, device, tuple(x.shape), x.device))
    st, sh, sd = x.stride()
    if sd != 1 or (sh != shape[2] and shape[1] > 1) or (st % 8 and shape[0] > 1) or x.data_ptr() % 16:
        x = x.contiguous()
        st = shape[1] * shape[2]
    return x, (st if shape[0] > 1 else shape[1] * shape[2])


def rope_append(cache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                slots: torch.Tensor, inv_freq: Optional[torch.Tensor] = None,
                q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                eps: float = 1e-6, interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                ws: Optional[Workspace] = None, stream=None) -> torch.Tensor:
    """Per-head RMS norm (where a weight is given) and rotary positions of a
    step's queries and keys, and the store of keys and values into ``cache``, a
    PagedCache or a PagedCache4 (``sa_rope_append``, ``sa_rope_append_kv4``).
    q [T][Hq][d], k and v [T][Hkv][d] bf16; positions int32 [T]; slots int64 [T]
    (-1: not stored); inv_freq fp32 [rot_dim / 2], None for no rotation.  Returns
    the queries, bf16 [T][Hq][d] (in ``q_out`` if given, which may be ``q``)."""
    if q_out is None:
        way = _short(ws, q.device, stream)
        if way is not None:
            fast, wp, wn, raw, _ = way
            four = isinstance(cache, PagedCache4)
            got = fast.append(cache.kv if four else cache.k, None if four else cache.v, cache.page_table,
                              cache.seq_lens, q, k, v, positions, slots, inv_freq, q_weight, k_weight, eps, interleaved,
                              wp, wn, raw)
            if got is not None:
                if isinstance(got, int):
                    _check(got, "sa_rope_append_kv4" if four else "sa_rope_append")
                return got
    return _rope_append(cache, q, k, v, positions, slots, inv_freq, q_weight, k_weight, eps, interleaved, q_out, ws,
                        stream=stream)


@_on_call_device
def _rope_append(cache, q, k, v, positions, slots, inv_freq, q_weight, k_weight, eps, interleaved, q_out, ws,
                 stream=None) -> torch.Tensor:
    four = isinstance(cache, PagedCache4)
    dev = q.device
    if q.dim() != 3:
        raise ValueError("rope_append: q must be bf16 [T][Hq][d], got shape %s" % (tuple(q.shape),))
    T, Hq, d = q.shape
    kv = kv4_struct(cache, dev) if four else kv_struct(cache, dev)
    if d != kv.head_dim:
        raise ValueError("rope_append: head_dim %d, the cache's is %d" % (d, kv.head_dim))
    if q_out is not None and q_out is not q:
        if q_out.dtype != torch.bfloat16 or tuple(q_out.shape) != (T, Hq, d) or q_out.device != dev or \
                q_out.stride(2) != 1 or q_out.stride(1) != d or q_out.stride(0) % 8 or q_out.data_ptr() % 16:
            raise ValueError("rope_append q_out: need a bf16 [T][Hq][d] tensor on %s with contiguous heads" % dev)
    src, qs = _rows(q, "q", (T, Hq, d), dev)
    if q_out is q and src is not q:
        raise ValueError("rope_append q_out: q is not laid out for an update in place")
    k, ks = _rows(k, "k", (T, kv.num_kv_heads, d), dev)
    v, vs = _rows(v, "v", (T, kv.num_kv_heads, d), dev)
    _need(positions, (T,), torch.int32, dev, "rope_append positions")
    _need(slots, (T,), torch.int64, dev, "rope_append slots")
    rot = 0
    if inv_freq is not None:
        _need(inv_freq, (inv_freq.numel(),), torch.float32, dev, "rope_append inv_freq")
        rot = 2 * inv_freq.numel()
    wt = torch.bfloat16
    for w, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            wt = w.dtype
            if wt not in (torch.bfloat16, torch.float32):
                raise TypeError("rope_append: %s must be bf16 or fp32, got %s" % (what, wt))
            _need(w, (d,), wt, dev, "rope_append " + what)
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise TypeError("rope_append: q_weight and k_weight must be of one type")
    if q_out is None:
        q_out = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=dev)
    a = L.AppendArgsS(src.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, q_out.data_ptr(),
                      q_out.stride(0) if T > 1 else Hq * d, positions.data_ptr(), slots.data_ptr(),
                      None if rot == 0 else inv_freq.data_ptr(), None if q_weight is None else q_weight.data_ptr(),
                      None if k_weight is None else k_weight.data_ptr(), L.DTYPE_F32 if wt == torch.float32 else
                      L.DTYPE_BF16, eps, T, Hq, rot, int(interleaved))
    wp, wn, raw, _ = _scratch(ws, dev, stream, 256)
    lib = L.load()
    fn = lib.sa_rope_append_kv4 if four else lib.sa_rope_append
    _check(fn(ctypes.byref(kv), ctypes.byref(a), wp, wn, raw),
           "sa_rope_append_kv4" if four else "sa_rope_append")
    return q_out


def expand_kv4(cache: PagedCache4, pages: torch.Tensor, k: Optional[torch.Tensor] = None,
               v: Optional[torch.Tensor] = None, ws: Optional[Workspace] = None, stream=None):
    """Pages of a 4-bit cache as bf16 pages (``sa_expand_kv4``): ``pages`` int32
    [n] (-1: that output page is left as it was) -> (k, v) bf16 [n][Hkv][P][d],
    pools that a PagedCache can hold."""
    if k is None and v is None:
        way = _short(ws, pages.device, stream)
        if way is not None:
            fast, wp, wn, raw, _ = way
            got = fast.expand(cache.kv, cache.page_table, cache.seq_lens, pages, wp, wn, raw)
            if got is not None:
                if isinstance(got, int):
                    _check(got, "sa_expand_kv4")
                return got
    return _expand_kv4(cache, pages, k, v, ws, stream=stream)


@_on_call_device
def _expand_kv4(cache, pages, k, v, ws, stream=None):
    dev = cache.kv.device
    kv = kv4_struct(cache)
    shape = (pages.numel(), kv.num_kv_heads, kv.page_size, kv.head_dim)
    _need(pages, (pages.numel(),), torch.int32, dev, "expand_kv4 pages")
    if k is None:
        k = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    else:
        _need(k, shape, torch.bfloat16, dev, "expand_kv4 k")
    if v is None:
        v = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    else:
        _need(v, shape, torch.bfloat16, dev, "expand_kv4 v")
    wp, wn, raw, _ = _scratch(ws, dev, stream, 256)
    _check(L.load().sa_expand_kv4(ctypes.byref(kv), pages.data_ptr(), shape[0], k.data_ptr(), v.data_ptr(), wp, wn,
                                  raw), "sa_expand_kv4")
    return k, v


@_on_call_stream
def check_bounded_wait(timeout_s: float, device=None, ws: Optional[Workspace] = None, stream=None) -> None:
    """Enqueue the bounded-wait diagnostic (``sa_check_bounded_wait``): a wait
    on an mbarrier that nothing arrives on gives up after ``timeout_s`` and
    records SA_ERR_TIMEOUT in the workspace, which ``ws.status()`` then reads."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    w = _ws(ws, dev, stream)
    wp, wn = w.aligned(256, stream)
    _check(L.load().sa_check_bounded_wait(int(timeout_s * 1e9), wp, wn, _stream(stream)), "sa_check_bounded_wait")


@_on_call_stream
def fetch_pages(host_k: torch.Tensor, host_v: torch.Tensor, dev_k: torch.Tensor, dev_v: torch.Tensor,
                pairs: torch.Tensor, ws: Optional[Workspace] = None, stream=None) -> None:
    """Copy host-tier pages into device page slots (``sa_fetch_pages``).
    host_k/host_v: pinned CPU tensors [host_pages][Hkv][P][d] bf16; dev_k/dev_v:
    device pools [slots][Hkv][P][d]; pairs: device int32 [n][2] {host page, slot}."""
    if not (host_k.is_pinned() and host_v.is_pinned()):
        raise ValueError("the host tier must be pinned memory")
    if host_k.shape[1:] != dev_k.shape[1:] or host_v.shape != host_k.shape or dev_v.shape != dev_k.shape:
        raise ValueError("host tier and device pool pages differ in shape")
    if host_k.dtype != torch.bfloat16 or dev_k.dtype != torch.bfloat16 or host_v.dtype != torch.bfloat16 \
            or dev_v.dtype != torch.bfloat16:
        raise ValueError("KV pages are bf16")
    if pairs.dtype != torch.int32 or pairs.dim() != 2 or pairs.shape[1] != 2 or not pairs.is_contiguous():
        raise ValueError("pairs must be a contiguous int32 [n][2] tensor")
    page_bytes = host_k[0].numel() * 2 if host_k.shape[0] else dev_k[0].numel() * 2
    w = _ws(ws, dev_k.device, stream)
    wp, wn = w.aligned(256, stream)
    _check(L.load().sa_fetch_pages(host_k.data_ptr(), host_v.data_ptr(), dev_k.data_ptr(), dev_v.data_ptr(),
                                   pairs.data_ptr(), pairs.shape[0], host_k.shape[0], dev_k.shape[0], page_bytes,
                                   wp, wn, _stream(stream)), "sa_fetch_pages")


@_on_call_stream
def select_blocks_spans(cache, spans: torch.Tensor, span_counts: torch.Tensor, span_round: torch.Tensor,
                        max_blocks: Optional[int] = None, out: Optional[BlockSelection] = None,
                        ws: Optional[Workspace] = None, stream=None) -> BlockSelection:
    """Span masks -> page-segment block list (``sa_select_blocks``, mode SPANS).
    spans int32 [B][max_spans][2], span_counts int32 [B], span_round uint8 [B][max_spans]."""
    B = cache.page_table.shape[0]
    dev = spans.device
    if out is None:
        mb = max_blocks if max_blocks is not None else cache.page_table.shape[1] + spans.shape[1]
        out = BlockSelection(torch.empty((B, mb, 4), dtype=torch.int32, device=dev),
                             torch.empty((B,), dtype=torch.int32, device=dev))
    _need(out.blocks, (B, out.blocks.shape[1], 4), torch.int32, dev, "select_blocks_spans out.blocks")
    _need(out.block_counts, (B,), torch.int32, dev, "select_blocks_spans out.block_counts")
    S = spans.shape[1]
    _need(spans, (B, S, 2), torch.int32, dev, "select_blocks_spans spans")
    _need(span_counts, (B,), torch.int32, dev, "select_blocks_spans span_counts")
    if span_round.dtype == torch.bool:
        span_round = span_round.to(torch.uint8)
    _need(span_round, (B, S), torch.uint8, dev, "select_blocks_spans span_round")
    kv = _geometry(cache, dev)
    a = L.BlockSelectArgsS()
    a.mode = L.SEL_SPANS
    a.spans, a.span_counts, a.span_round = spans.data_ptr(), span_counts.data_ptr(), span_round.data_ptr()
    a.max_spans = spans.shape[1]
    o = L.BlockListS()
    o.blocks, o.block_counts, o.max_blocks = out.blocks.data_ptr(), out.block_counts.data_ptr(), out.blocks.shape[1]
    w = _ws(ws, dev, stream)
    wp, wn = w.aligned(workspace_bytes(L.OP_SELECT_BLOCKS, cache, block_args=a), stream)
    _check(L.load().sa_select_blocks(ctypes.byref(kv), ctypes.byref(a), ctypes.byref(o), wp, wn,
                                     _stream(stream)), "sa_select_blocks(spans)")
    return out


@_on_call_stream
def select_blocks_rbs(cache, q: torch.Tensor, block_size: int = 64, scale: Optional[float] = None,
                      tau_c=None, tau_r=None, p_c: float = 0.95, p_r: float = 0.97,
                      force_diag: bool = True, force_first: bool = True,
                      nnz_capacity: Optional[int] = None, out: Optional[BlockCSR] = None,
                      ws: Optional[Workspace] = None, stream=None) -> BlockCSR:
    """RBS two-branch block selection (``sa_select_blocks``, mode RBS).
    Explicit thresholds: tau_c / tau_r fp32 [Hq] tensors (or floats);
    otherwise quantile mode with p_c / p_r."""
    T, Hq, d = q.shape
    dev = q.device
    q = _bf16_q(q, "select_blocks_rbs")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    nB = (T + block_size - 1) // block_size
    if out is None:
        cap = nnz_capacity if nnz_capacity is not None else Hq * nB * (nB + 1) // 2
        out = BlockCSR(torch.empty(Hq * nB + 1, dtype=torch.int32, device=dev),
                       torch.empty(max(cap, 1), dtype=torch.int32, device=dev),
                       torch.empty((2, Hq), dtype=torch.float32, device=dev), Hq, nB)
    _need(out.row_ptr, (Hq * nB + 1,), torch.int32, dev, "select_blocks_rbs out.row_ptr")
    _need(out.cols, (out.cols.numel(),), torch.int32, dev, "select_blocks_rbs out.cols")
    _need(out.tau, (2, Hq), torch.float32, dev, "select_blocks_rbs out.tau")
    tc = tr = None
    if tau_c is not None:
        tc = torch.as_tensor(tau_c, dtype=torch.float32, device=dev).expand(Hq).contiguous()
        tr = torch.as_tensor(tau_r, dtype=torch.float32, device=dev).expand(Hq).contiguous()
    kv = kv_struct(cache, dev)
    a = L.BlockSelectArgsS()
    a.mode = L.SEL_RBS
    a.q = q.data_ptr()
    a.num_q_heads, a.num_tokens, a.block_size, a.scale = Hq, T, block_size, scale
    a.tau_c = None if tc is None else tc.data_ptr()
    a.tau_r = None if tr is None else tr.data_ptr()
    a.p_c, a.p_r = p_c, p_r
    a.force_diag, a.force_first = int(force_diag), int(force_first)
    o = L.BlockListS()
    o.row_ptr, o.cols, o.nnz_capacity = out.row_ptr.data_ptr(), out.cols.data_ptr(), out.cols.numel()
    o.tau_out = out.tau.data_ptr()
    w = _ws(ws, dev, stream)
    wp, wn = w.aligned(workspace_bytes(L.OP_SELECT_BLOCKS, cache, block_args=a), stream)
    _check(L.load().sa_select_blocks(ctypes.byref(kv), ctypes.byref(a), ctypes.byref(o), wp, wn,
                                     _stream(stream)), "sa_select_blocks(rbs)")
    return out


@_on_call_stream
def sparse_prefill_attn(cache, q: torch.Tensor, csr: BlockCSR, scale: Optional[float] = None,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        want_lse: bool = True, ws: Optional[Workspace] = None, stream=None):
    """Causal block-sparse prefill (``sa_sparse_prefill_attn``).  Returns (out bf16, lse fp32)."""
    T, Hq, d = q.shape
    dev = q.device
    q = _bf16_q(q, "sparse_prefill_attn")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=dev)
    _need(out, (T, Hq, d), torch.bfloat16, dev, "sparse_prefill_attn out")
    if lse is None and want_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    if lse is not None:
        _need(lse, (T, Hq), torch.float32, dev, "sparse_prefill_attn lse")
    nQB = (T + 63) // 64
    _need(csr.row_ptr, (Hq * nQB + 1,), torch.int32, dev, "sparse_prefill_attn csr.row_ptr")
    _need(csr.cols, (csr.cols.numel(),), torch.int32, dev, "sparse_prefill_attn csr.cols")
    kv = kv_struct(cache, dev)
    c = L.BlockListS()
    c.row_ptr, c.cols, c.nnz_capacity = csr.row_ptr.data_ptr(), csr.cols.data_ptr(), csr.cols.numel()
    w = _ws(ws, dev, stream)
    wp, wn = w.aligned(workspace_bytes(L.OP_PREFILL, cache, num_q_heads=Hq, num_tokens=T), stream)
    _check(L.load().sa_sparse_prefill_attn(ctypes.byref(kv), _ptr(q), Hq, T, ctypes.byref(c), scale, 1,
                                           _ptr(out), _ptr(lse), wp, wn, _stream(stream)),
           "sa_sparse_prefill_attn")
    return out, lse
