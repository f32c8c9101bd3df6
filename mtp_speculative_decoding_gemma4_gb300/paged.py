"""Torch-facing layer over the paged-cache entry points of the C ABI: the cache's descriptor,
argument checks and output allocation. Marshalling only; every operator runs in libmtp.so.

Outputs and workspaces come from torch's allocator on the stream that the call uses: by default
torch's current stream of the tensors' device, else the cudaStream_t passed as `stream`.
"""
from __future__ import annotations

import ctypes
import threading
from typing import Optional

import torch

from . import binding as B

_DT = {torch.bfloat16: B.MTP_DTYPE_BF16, torch.float32: B.MTP_DTYPE_F32}


_i32, _f32 = torch.int32, torch.float32


def _flat_like(t, dtype, device, shape) -> bool:
    """Whether t is what _need_flat asks for; the common case of a check, without its message."""
    return isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.shape == shape and \
        t.is_contiguous()


def _need(t, name: str, dtype, ndim: int, device=None) -> torch.Tensor:
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.dim() == ndim):
        raise ValueError(f"{name} must be a {ndim}-dimensional CUDA tensor of {dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    return t


def _need_flat(t, name: str, dtype, shape, device=None) -> torch.Tensor:
    _need(t, name, dtype, len(shape), device)
    ok = t.is_contiguous()
    for n, m in zip(shape, t.shape):
        ok = ok and (n is None or n == m)
    if not ok:
        raise ValueError(f"{name} must be contiguous of shape {list(shape)} (got {list(t.shape)})")
    return t


class _On:
    """A call's device and stream where they are not the current ones: makes the tensors' device
    current and allocates on the given stream."""

    def __init__(self, device: torch.device, stream: Optional[int]):
        self._ctx = [torch.cuda.device(device)]
        if stream is not None:
            self._ctx.append(torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if stream else
                                               torch.cuda.default_stream(device)))
        self._device, self._stream = device, stream

    def __enter__(self) -> int:
        for c in self._ctx:
            c.__enter__()
        return _raw_stream(self._device.index) if self._stream is None else self._stream

    def __exit__(self, *exc):
        for c in reversed(self._ctx):
            c.__exit__(*exc)


_raw_stream = torch._C._cuda_getCurrentRawStream  # torch's current stream of a device, as an integer
_current_device = torch._C._cuda_getDevice


def call_on(device: torch.device, stream: Optional[int], fn, *args):
    """fn(stream, *args) with the call's device current and its allocations on its stream."""
    index = device.index
    if _current_device() == index:
        current = _raw_stream(index)
        if stream is None or stream == current:
            return fn(current, *args)
    with _On(device, stream) as st:
        return fn(st, *args)


class PagedKV:
    """A key cache in pages: k [n_pages][P][n_kv][d] (bf16 or fp32, last dimension contiguous;
    other strides free, so a head-major cache is passed as its transposed view), v of the same
    strides or None (V = K), block_table int32 [B][max_pages], ctx_len int32 [B]; codes int8
    [n_pages][n_kv][d] and scales fp32 [n_pages][n_kv] hold page summaries (page_append writes
    them, page_select scores them). block_table and ctx_len may be None for page_append alone.
    Holds the tensors; the descriptor is made once and the buffers may change their contents."""

    def __init__(self, k: torch.Tensor, block_table: Optional[torch.Tensor] = None,
                 ctx_len: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                 codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None):
        if not (isinstance(k, torch.Tensor) and k.is_cuda and k.dtype in _DT and k.dim() == 4):
            raise ValueError("k must be a 4-dimensional CUDA tensor [n_pages][P][n_kv][d] of bf16 or fp32")
        dev = k.device
        n_pages, P, n_kv, d = k.shape
        if v is not None:
            _need(v, "v", k.dtype, 4, dev)
            if v.shape != k.shape or v.stride() != k.stride():
                raise ValueError("v must have the shape and strides of k")
        if k.stride(3) != 1:
            raise ValueError("the last dimension of k must be contiguous")
        c = self.c = B.mtp_paged_kv()
        if block_table is not None:
            _need(block_table, "block_table", torch.int32, 2, dev)
            if block_table.shape[1] > 1 and block_table.stride(1) != 1:
                raise ValueError("the last dimension of block_table must be contiguous")
            if ctx_len is None:
                raise ValueError("block_table needs ctx_len")
            _need_flat(ctx_len, "ctx_len", torch.int32, (block_table.shape[0],), dev)
            c.block_table, c.ctx_len = block_table.data_ptr(), ctx_len.data_ptr()
            c.max_pages = block_table.shape[1]
            c.table_stride = block_table.stride(0) if block_table.shape[0] > 1 else block_table.shape[1]
        if codes is not None or scales is not None:
            _need_flat(codes, "codes", torch.int8, (n_pages, n_kv, d), dev)
            _need_flat(scales, "scales", torch.float32, (n_pages, n_kv), dev)
            c.codes, c.scales = codes.data_ptr(), scales.data_ptr()
        c.k, c.v = k.data_ptr(), 0 if v is None else v.data_ptr()
        # the stride of a dimension of size one is never used: any legal value
        c.stride_page = k.stride(0) if n_pages > 1 else max(k.stride(0), P * n_kv * d)
        c.stride_t = k.stride(1) if P > 1 else max(k.stride(1), n_kv * d)
        c.stride_h = k.stride(2) if n_kv > 1 else d
        c.n_pages, c.page_size, c.n_kv_head, c.head_dim, c.dtype = n_pages, P, n_kv, d, _DT[k.dtype]
        self.k, self.v, self.block_table, self.ctx_len, self.codes, self.scales = k, v, block_table, ctx_len, codes, scales
        self.device, self.batch = dev, 0 if block_table is None else block_table.shape[0]
        self._row = (n_kv, d)
        self.p = ctypes.byref(c)  # the descriptor as the C entry points take it
        self._ws = {}  # workspace bytes by (n_head, n_list); and of the selection by "select"
        self._scratch, self._scratch_at, self._scratch_n, self._lock = None, 0, 0, threading.Lock()


def _with_workspace(kv: PagedKV, st: int, n: int, launch) -> None:
    """launch(pointer, n) with a workspace of n bytes for a call on stream st. The default stream's
    calls on a cache follow one another (and are never captured), so they share one buffer kept with
    the descriptor, under a lock that keeps the launches of a call together: an allocation costs 3 us
    of a call's 17 on the host. Any other stream's calls get a buffer of their own."""
    if not n:
        launch(0, 0)
    elif st != 0:
        ws = torch.empty(n, dtype=torch.uint8, device=kv.device)
        launch(ws.data_ptr(), n)
    else:
        with kv._lock:
            if kv._scratch_n < n:
                kv._scratch = torch.empty(n, dtype=torch.uint8, device=kv.device)
                kv._scratch_at, kv._scratch_n = kv._scratch.data_ptr(), n
            launch(kv._scratch_at, n)


def page_plan(old_len: torch.Tensor, new_len: torch.Tensor, block_table: torch.Tensor, free_ring: torch.Tensor,
              ring_state: torch.Tensor, page_size: int, max_tokens: int, stream: Optional[int] = None):
    """Takes and returns pages so that sequence b holds new_len[b] instead of old_len[b] tokens
    (int32 [B]): updates block_table [B][max_pages] and the ring of free pages free_ring
    [n_pages] (ring_state: head and count) in place and returns (len_out [B], slot_map
    [max_tokens], cu_new [B + 1], state_out [2], status [4]), as mtp_page_plan describes."""
    _need_flat(old_len, "old_len", _i32, (None,))
    dev, shape = old_len.device, old_len.shape
    Bn = shape[0]
    if not _flat_like(new_len, _i32, dev, shape):
        _need_flat(new_len, "new_len", _i32, shape, dev)
    _need(block_table, "block_table", _i32, 2, dev)
    _need_flat(free_ring, "free_ring", _i32, (None,), dev)
    if not _flat_like(ring_state, _i32, dev, (2,)):
        _need_flat(ring_state, "ring_state", _i32, (2,), dev)
    if block_table.shape[0] != Bn or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError(f"block_table must be [{Bn}][max_pages] with a contiguous last dimension")
    if max_tokens < 0:
        raise ValueError("max_tokens must be >= 0")
    return call_on(dev, stream, _plan, old_len, new_len, block_table, free_ring, ring_state, page_size, max_tokens)


def _plan(st, old_len, new_len, block_table, free_ring, ring_state, page_size, max_tokens):
    (Bn, cols), dev, i32 = block_table.shape, old_len.device, _i32
    len_out = torch.empty_like(old_len)
    slots = torch.empty(max_tokens, dtype=i32, device=dev)
    cu = torch.empty(Bn + 1, dtype=i32, device=dev)
    state = torch.empty_like(ring_state)
    status = torch.empty(4, dtype=i32, device=dev)
    B.mtp_page_plan(old_len.data_ptr(), new_len.data_ptr(), Bn, block_table.data_ptr(),
                    block_table.stride(0) if Bn > 1 else cols, cols, free_ring.data_ptr(), free_ring.shape[0],
                    ring_state.data_ptr(), page_size, max_tokens, len_out.data_ptr(), slots.data_ptr(), cu.data_ptr(),
                    state.data_ptr(), status.data_ptr(), st)
    return len_out, slots, cu, state, status


def page_append(kv: PagedKV, k_new: torch.Tensor, slot_map: torch.Tensor, v_new: Optional[torch.Tensor] = None,
                stream: Optional[int] = None) -> None:
    """Writes row t of k_new [T][n_kv][d] (and v_new, for a cache with a V) into slot slot_map[t]
    (int32 [T]; slots outside the cache are skipped) and, for a cache with summaries, refreshes
    the summary of every page whose last slot is written. Rows may be strided (the last two
    dimensions contiguous)."""
    n_kv, d = kv._row
    for t, name in ((k_new, "k_new"), (v_new, "v_new")):
        if t is None:
            continue
        _need(t, name, kv.k.dtype, 3, kv.device)
        T = k_new.shape[0]
        if t.shape != (T, n_kv, d) or T and (t.stride(2) != 1 or n_kv > 1 and t.stride(1) != d):
            raise ValueError(f"{name} must be [T][{n_kv}][{d}] with contiguous rows")
    if not _flat_like(slot_map, _i32, kv.device, k_new.shape[:1]):
        _need_flat(slot_map, "slot_map", _i32, (k_new.shape[0],), kv.device)
    call_on(kv.device, stream, _append, kv, k_new, slot_map, v_new)


def _append(st, kv, k_new, slot_map, v_new):
    T, width = k_new.shape[0], kv.c.n_kv_head * kv.c.head_dim
    B.mtp_page_append(kv.p, k_new.data_ptr(), 0 if v_new is None else v_new.data_ptr(),
                      k_new.stride(0) if T > 1 else width, v_new.stride(0) if T > 1 and v_new is not None else width,
                      slot_map.data_ptr(), T, st)


def page_fork(kv: PagedKV, src: torch.Tensor, dst: torch.Tensor, length: torch.Tensor, free_ring: torch.Tensor,
              ring_state: torch.Tensor, stream: Optional[int] = None):
    """Makes sequences dst[i] copies of the first length[i] tokens of sequences src[i] (int32 [n]):
    complete pages are shared through kv's block_table (updated in place), a partial page's rows are
    copied into a page from the ring of free pages free_ring [n_pages] (ring_state: head and count).
    Returns (len_out [B], state_out [2], status [4]), as mtp_page_fork describes, with what sharing
    pages asks of a program."""
    if kv.block_table is None:
        raise ValueError("the cache has no block_table")
    dev = kv.device
    _need_flat(src, "src", _i32, (None,), dev)
    for t, name, shape in ((dst, "dst", src.shape), (length, "length", src.shape), (ring_state, "ring_state", (2,)),
                           (free_ring, "free_ring", (kv.c.n_pages,))):
        if not _flat_like(t, _i32, dev, shape):
            _need_flat(t, name, _i32, shape, dev)
    return call_on(dev, stream, _fork, kv, src, dst, length, free_ring, ring_state)


def _fork(st, kv, src, dst, length, free_ring, ring_state):
    len_out, state, dev = torch.empty_like(kv.ctx_len), torch.empty_like(ring_state), kv.device
    status = torch.empty(4, dtype=_i32, device=dev)
    B.mtp_page_fork(kv.p, kv.batch, src.data_ptr(), dst.data_ptr(), length.data_ptr(), src.shape[0], free_ring.data_ptr(),
                    ring_state.data_ptr(), len_out.data_ptr(), state.data_ptr(), status.data_ptr(), st)
    return len_out, state, status


def page_collect(kv: PagedKV, free_ring: torch.Tensor, compact: bool = False, stream: Optional[int] = None):
    """Makes the pages that no sequence of kv holds the ring of free pages (free_ring [n_pages], from
    its beginning), whatever held them before; with compact, moves the held pages into the front of
    the pool first. Returns (table_out, state_out [2], status [4]), as mtp_page_collect describes:
    table_out [B][max_pages] under the pages' new numbers with compact, else None."""
    if kv.block_table is None:
        raise ValueError("the cache has no block_table")
    if not _flat_like(free_ring, _i32, kv.device, (kv.c.n_pages,)):
        _need_flat(free_ring, "free_ring", _i32, (kv.c.n_pages,), kv.device)
    return call_on(kv.device, stream, _collect, kv, free_ring, bool(compact))


def _collect(st, kv, free_ring, compact):
    n = kv._ws.get(("collect", compact))
    if n is None:
        n = kv._ws[("collect", compact)] = B.mtp_page_collect_workspace(kv.p, int(compact))
    cols = kv.c.max_pages
    table = torch.empty((kv.batch, cols), dtype=_i32, device=kv.device) if compact else None
    state, status = torch.empty(2, dtype=_i32, device=kv.device), torch.empty(4, dtype=_i32, device=kv.device)
    _with_workspace(kv, st, n, lambda ws, n: B.mtp_page_collect(
        kv.p, kv.batch, free_ring.data_ptr(), table.data_ptr() if compact else 0, cols, state.data_ptr(),
        status.data_ptr(), ws, n, st))
    return table, state, status


def _queries(q, kv: PagedKV):
    """Checks the queries; their shape."""
    shape = q.shape if isinstance(q, torch.Tensor) else ()
    if not (len(shape) == 3 and shape[0] == kv.batch and shape[2] == kv._row[1] and
            _flat_like(q, _f32, kv.device, shape)):
        _need_flat(q, "q", _f32, (kv.batch, None, kv._row[1]), kv.device)
    if kv.block_table is None:
        raise ValueError("the cache has no block_table")
    return shape


def paged_attention(q: torch.Tensor, kv: PagedKV, window: int = 0, scale: float = 0.0,
                    pages: Optional[torch.Tensor] = None, want_lse: bool = False, out: Optional[torch.Tensor] = None,
                    stream: Optional[int] = None):
    """Attention of one new token per sequence, q fp32 [B][n_head][d], over the paged cache: all
    ctx_len[b] keys, the last `window` (> 0), or those of the logical pages listed in `pages`
    (int32 [B][n_kv][n], -1: none). Returns out fp32 [B][n_head][d], with want_lse (out, lse
    [B][n_head])."""
    shape, n_list = _queries(q, kv), 0
    if pages is not None:
        _need_flat(pages, "pages", _i32, (kv.batch, kv._row[0], None), kv.device)
        n_list = pages.shape[2]
        if n_list < 1:
            raise ValueError("pages must list at least one entry per KV head")
    if out is not None:
        _need_flat(out, "out", _f32, shape, kv.device)
    return call_on(kv.device, stream, _attend, q, kv, shape[0], shape[1], window, scale, pages, n_list, want_lse, out)


def _attend(st, q, kv, Bn, nh, window, scale, pages, n_list, want_lse, out):
    n = kv._ws.get((nh, n_list))
    if n is None:
        n = kv._ws[(nh, n_list)] = B.mtp_paged_attention_workspace(kv.p, Bn, nh, n_list)
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty((Bn, nh), dtype=_f32, device=kv.device) if want_lse else None
    _with_workspace(kv, st, n, lambda ws, n: B.mtp_paged_attention(
        kv.p, q.data_ptr(), Bn, nh, window, scale, 0 if pages is None else pages.data_ptr(), n_list, out.data_ptr(),
        lse.data_ptr() if want_lse else 0, ws, n, st))
    return (out, lse) if want_lse else out


def paged_attention_chunk(q: torch.Tensor, kv: PagedKV, cu_new: torch.Tensor, window: int = 0, scale: float = 0.0,
                          want_lse: bool = False, out: Optional[torch.Tensor] = None, stream: Optional[int] = None):
    """Attention of the new tokens of every sequence, q [T][n_head][d] of the cache's dtype, over the
    paged cache, which holds their keys already: rows [cu_new[b], cu_new[b + 1]) (int32 [B + 1]) are
    the last tokens of sequence b, and each attends the keys up to its own position, the last `window`
    of them where that is > 0. Rows may be strided (the last two dimensions contiguous). Returns out
    [T][n_head][d] (q's dtype), with want_lse (out, lse fp32 [T][n_head]). Rows of no sequence are
    left as they were, unset in tensors that the call allocates."""
    if kv.block_table is None:
        raise ValueError("the cache has no block_table")
    _need(q, "q", kv.k.dtype, 3, kv.device)
    T, nh, d = q.shape
    if d != kv._row[1] or T and (q.stride(2) != 1 or nh > 1 and q.stride(1) != d):
        raise ValueError(f"q must be [T][n_head][{kv._row[1]}] with contiguous rows (got {list(q.shape)})")
    if not _flat_like(cu_new, _i32, kv.device, (kv.batch + 1,)):
        _need_flat(cu_new, "cu_new", _i32, (kv.batch + 1,), kv.device)
    if out is not None:
        _need_flat(out, "out", q.dtype, q.shape, kv.device)
    return call_on(kv.device, stream, _attend_chunk, q, kv, cu_new, window, scale, want_lse, out)


def _attend_chunk(st, q, kv, cu_new, window, scale, want_lse, out):
    T, nh, d = q.shape
    n = kv._ws.get(("chunk", T, nh))
    if n is None:
        if len(kv._ws) >= 1024:  # (calls of many lengths)
            kv._ws.clear()
        n = kv._ws[("chunk", T, nh)] = B.mtp_paged_attention_chunk_workspace(kv.p, kv.batch, T, nh)
    if out is None:
        out = torch.empty((T, nh, d), dtype=q.dtype, device=kv.device)
    lse = torch.empty((T, nh), dtype=_f32, device=kv.device) if want_lse else None
    _with_workspace(kv, st, n, lambda ws, n: B.mtp_paged_attention_chunk(
        kv.p, q.data_ptr(), q.stride(0) if T > 1 else nh * d, cu_new.data_ptr(), kv.batch, T, nh, window, scale,
        out.data_ptr(), lse.data_ptr() if want_lse else 0, ws, n, st))
    return (out, lse) if want_lse else out


def page_select(q: torch.Tensor, kv: PagedKV, n_select: int, keep_first: int = 1, keep_last: int = 1,
                out: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> torch.Tensor:
    """The n_select logical pages of the highest scores per sequence and KV head, in increasing
    order (int32 [B][n_kv][n_select], -1 behind them): the first keep_first and last keep_last
    pages, then those whose summaries' dot product with q is largest. A list for
    paged_attention(pages=...)."""
    Bn, nh, _ = _queries(q, kv)
    if n_select < 1:
        raise ValueError("n_select must be >= 1")
    if out is not None:
        _need_flat(out, "out", _i32, (kv.batch, kv._row[0], n_select), kv.device)
    return call_on(kv.device, stream, _select, q, kv, Bn, nh, n_select, keep_first, keep_last, out)


def _select(st, q, kv, Bn, nh, n_select, keep_first, keep_last, out):
    if out is None:
        out = torch.empty((Bn, kv._row[0], n_select), dtype=_i32, device=kv.device)
    n = kv._ws.get("select")
    if n is None:
        n = kv._ws["select"] = B.mtp_page_select_workspace(kv.p, Bn)
    _with_workspace(kv, st, n, lambda ws, n: B.mtp_page_select(
        kv.p, q.data_ptr(), Bn, nh, n_select, keep_first, keep_last, out.data_ptr(), ws, n, st))
    return out
