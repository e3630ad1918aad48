"""Paged serving calls: requests of different lengths over shared cache pages.

The binding of the paged section of ``include/hca.h``: a step's block tables
and slot maps from request lengths (``kv_page_plan``), the step's raw tokens
and pooled entries into their pages (``kv_page_store``, ``kv_page_compress``),
and attention of the new tokens over the pages (``paged_attn_chunk`` for HCA
layers, ``paged_attn_window`` for window-only layers).  All lengths stay on
the device.  Each call runs on the device of its tensors, on that device's
current stream unless ``stream`` is given.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from . import (_F, _I32, _I64, _SZ, _V, AttnExtrasStruct, CacheStruct, EntryExtrasStruct, KVCache, LAYOUT_128,
               LAYOUT_512, Layout, _check, _lib)

_NONE = contextlib.nullcontext()
_BF, _INT, _LONG, _FLOAT = torch.bfloat16, torch.int32, torch.int64, torch.float32


class PageMapStruct(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("width", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("pages", ctypes.c_int64)]


_EE, _AE = ctypes.POINTER(EntryExtrasStruct), ctypes.POINTER(AttnExtrasStruct)
_lib.kv_page_plan.argtypes = [_V, _V, _I32, _I32, _I32, _V, _I32, _V, _V, _I32, _I64, _V, _V, _V, _V, _V, _V, _V]
_lib.kv_page_plan.restype = ctypes.c_int
_lib.kv_page_store.argtypes = [_V, _I64, _V, _V, _V, Layout, _EE, _V, _I64, _V]
_lib.kv_page_store.restype = ctypes.c_int
_lib.kv_page_compress.argtypes = [_I32, _V, _V, _I64, _V, _V, _I32, _V, _V, _V, _V, _V, _I64, _V, _V, Layout,
                                  CacheStruct, _I64, _EE, _V]
_lib.kv_page_compress.restype = ctypes.c_int
_lib.paged_attn_workspace_size.argtypes = [_I64, _I32, _I32, Layout, _I64, _I64, _I32, _I32]
_lib.paged_attn_workspace_size.restype = _SZ
_lib.paged_attn_chunk.argtypes = [_V, _I64, _I32, _I32, _V, _V, _I64, _I32, Layout, CacheStruct, PageMapStruct, _V,
                                  PageMapStruct, _I32, _F, _AE, _V, _V, _SZ, _V]
_lib.paged_attn_chunk.restype = ctypes.c_int
_lib.paged_attn_window.argtypes = [_V, _I64, _I32, _I32, _V, _V, _I64, Layout, _V, PageMapStruct, _I32, _I32, _F, _AE,
                                   _V, _V, _SZ, _V]
_lib.paged_attn_window.restype = ctypes.c_int


def _ok(t, dt, shape, dev):
    """The usual case, decided in well under a microsecond."""
    return t.dtype is dt and t.shape == shape and t.is_contiguous() and t.device == dev


def _want(dev, *specs):
    """Each (tensor, dtype, shape, name): contiguous, on `dev`, of that dtype
    and shape (None: any extent)."""
    for t, dt, shape, name in specs:
        if t.dtype != dt:
            raise TypeError(f"{name}: expected {dt}, got {t.dtype}")
        if t.device != dev:
            raise ValueError(f"{name}: must be on {dev}, is on {t.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
        s = t.shape
        if len(s) != len(shape) or any(w is not None and w != h for w, h in zip(shape, s)):
            raise ValueError(f"{name}: expected shape {shape}, got {tuple(s)}")


def _device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    return t.device


def _on(dev):
    """The device of the call's tensors made current (the launches go there)."""
    return _NONE if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


# the current stream's handle without building a Stream object, where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _st(dev, stream):
    if stream is None:
        return _raw_stream(dev.index)
    if stream.device != dev:
        raise ValueError(f"stream: must be of {dev}, is of {stream.device}")
    return stream.cuda_stream


_LAYOUT = {(512, 64, 64): Layout(512, 64, 64), (128, 32, 32): Layout(128, 32, 32)}


def _layout(layout):
    return _LAYOUT.get(tuple(layout)) or Layout(*layout)


def _entry_extras(extras, layout, dev):
    if extras is None:
        return None
    if extras.norm_w is not None and not _ok(extras.norm_w, _FLOAT, (layout[0],), dev):
        _want(dev, (extras.norm_w, _FLOAT, (layout[0],), "norm_w"))
    if extras.inv_freq is not None and not _ok(extras.inv_freq, _FLOAT, (layout[1] // 2,), dev):
        _want(dev, (extras.inv_freq, _FLOAT, (layout[1] // 2,), "inv_freq"))
    return ctypes.byref(extras.c_struct())


class PagePlan:
    """A step's plan (kv_page_plan): row_start int32 [B+1]; row_req, row_pos
    int32 [max_rows]; slot int64 [max_rows]; missing, free_left int32 [1]."""

    __slots__ = ("row_start", "row_req", "row_pos", "slot", "missing", "free_left")

    def __init__(self, row_start, row_req, row_pos, slot, missing=None, free_left=None):
        self.row_start, self.row_req, self.row_pos, self.slot = row_start, row_req, row_pos, slot
        self.missing, self.free_left = missing, free_left

    @classmethod
    def empty(cls, B: int, max_rows: int, device="cuda") -> "PagePlan":
        """Buffers of a plan of B requests and up to max_rows rows (row_req,
        row_pos and slot start at -1: rows past the last stay so)."""
        full = lambda n, dt: torch.full((n,), -1, dtype=dt, device=device)
        zero = lambda n: torch.zeros((n,), dtype=_INT, device=device)
        return cls(zero(B + 1), full(max_rows, _INT), full(max_rows, _INT), full(max_rows, _LONG), zero(1), zero(1))

    def check(self, dev, B=None, totals=False):
        """The buffers' types, sizes (of B requests) and device; totals: missing
        and free_left, which kv_page_plan writes, too."""
        if totals:
            for t, name in ((self.missing, "plan.missing"), (self.free_left, "plan.free_left")):
                if t is None:
                    raise ValueError(f"{name}: is needed to make a plan (int32 [1])")
                if not _ok(t, _INT, (1,), dev):
                    _want(dev, (t, _INT, (1,), name))
        n = self.slot.shape[0]
        s = self.row_start
        if (_ok(self.slot, _LONG, (n,), dev) and _ok(self.row_pos, _INT, (n,), dev) and _ok(self.row_req, _INT, (n,), dev)
                and _ok(s, _INT, (s.shape[0] if B is None else B + 1,), dev) and s.shape[0] > 0):
            return
        _want(dev, (self.row_start, _INT, (None if B is None else B + 1,), "plan.row_start"),
              (self.row_req, _INT, (n,), "plan.row_req"), (self.row_pos, _INT, (n,), "plan.row_pos"),
              (self.slot, _LONG, (n,), "plan.slot"))
        if s.shape[0] == 0:                      # (its last element is the count of live rows)
            raise ValueError("plan.row_start: must hold B + 1 offsets")


def kv_page_plan(ctx_len, new_len, m: int, page_size: int, block_table, free_pages, free_count, plan=None,
                 max_rows=None, stream=None) -> PagePlan:
    """Block tables and slot maps of one step from request lengths: ctx_len,
    new_len int32 [B]; m = 1 for tokens, or tokens per entry; block_table int32
    [B][width] (updated in place with the step's fresh pages); free_pages int32
    stack with free_count int32 [1] numbers in use (neither is changed:
    plan.free_left is the next step's count).  plan: buffers to write
    (PagePlan.empty), or None with max_rows.  plan.missing counts pages that
    the step's rows need and do not have, now or since an earlier step; such
    rows have slot -1."""
    dev = _device(ctx_len, "ctx_len")
    B = ctx_len.shape[0]
    if plan is None:
        if max_rows is None:
            raise ValueError("kv_page_plan: give plan or max_rows")
        with _NONE if stream is None else torch.cuda.stream(stream):
            plan = PagePlan.empty(B, max_rows, dev)
    width, n_free = block_table.shape[-1], free_pages.shape[0]
    if not (_ok(ctx_len, _INT, (B,), dev) and _ok(new_len, _INT, (B,), dev) and _ok(block_table, _INT, (B, width), dev)
            and _ok(free_pages, _INT, (n_free,), dev) and _ok(free_count, _INT, (1,), dev)):
        _want(dev, (ctx_len, _INT, (B,), "ctx_len"), (new_len, _INT, (B,), "new_len"),
              (block_table, _INT, (B, None), "block_table"), (free_pages, _INT, (None,), "free_pages"),
              (free_count, _INT, (1,), "free_count"))
    plan.check(dev, B, totals=True)
    with _on(dev):
        _check(_lib.kv_page_plan(ctx_len.data_ptr(), new_len.data_ptr(), B, m, page_size, block_table.data_ptr(),
                                 width, free_pages.data_ptr(), free_count.data_ptr(),
                                 n_free, plan.slot.shape[0], plan.row_start.data_ptr(),
                                 plan.row_req.data_ptr(), plan.row_pos.data_ptr(), plan.slot.data_ptr(),
                                 plan.missing.data_ptr(), plan.free_left.data_ptr(), _st(dev, stream)), "kv_page_plan")
    return plan


def kv_page_store(x, plan: PagePlan, pages, layout, extras=None, stream=None):
    """The step's raw tokens x [n][d] bf16 into their pages [pages][page_size][d]
    (rows plan.row_start[B] .. are skipped; n <= the plan's rows).  extras: an
    EntryExtras (RMSNorm, RoPE at each token's position) or None (a copy)."""
    dev = _device(x, "x")
    n, d = x.shape[0], layout[0]
    np_, ps = pages.shape[0], pages.shape[-2]
    if not (_ok(x, _BF, (n, d), dev) and _ok(pages, _BF, (np_, ps, d), dev)):
        _want(dev, (x, _BF, (None, d), "x"), (pages, _BF, (None, None, d), "pages"))
    plan.check(dev)
    if n > plan.slot.shape[0]:
        raise ValueError("x: more rows than the plan holds")
    with _on(dev):
        _check(_lib.kv_page_store(x.data_ptr(), n, plan.row_start.data_ptr() + 4 * (plan.row_start.shape[0] - 1),
                                  plan.row_pos.data_ptr(), plan.slot.data_ptr(), _layout(layout),
                                  _entry_extras(extras, layout, dev), pages.data_ptr(), np_ * ps, _st(dev, stream)),
               "kv_page_store")
    return pages


def kv_page_compress(x, gate, pos_bias, row_start, ctx_len, plan: PagePlan, tail_x, tail_gate, cache: KVCache,
                     extras=None, stream=None):
    """The blocks that the step completes, pooled into entry pages: x, gate
    [n][d] bf16 raw tokens (request b's at rows row_start[b] ..); pos_bias
    [m][d] (m = 4 or 128); plan: kv_page_plan with this m; tail_x, tail_gate
    [B][m][d] bf16, in and out: the incomplete block's tokens, token t in row
    t % m; cache: the entry pool (a KVCache of B = pages, capacity =
    page_size)."""
    dev = _device(x, "x")
    d, B, m = cache.layout[0], ctx_len.shape[0], pos_bias.shape[0]
    n = x.shape[0]
    if not (_ok(x, _BF, (n, d), dev) and _ok(gate, _BF, (n, d), dev) and _ok(pos_bias, _FLOAT, (m, d), dev)
            and _ok(row_start, _INT, (B + 1,), dev) and _ok(ctx_len, _INT, (B,), dev)
            and _ok(tail_x, _BF, (B, m, d), dev) and _ok(tail_gate, _BF, (B, m, d), dev)):
        _want(dev, (x, _BF, (n, d), "x"), (gate, _BF, (n, d), "gate"), (pos_bias, _FLOAT, (m, d), "pos_bias"),
              (row_start, _INT, (B + 1,), "row_start"), (ctx_len, _INT, (B,), "ctx_len"),
              (tail_x, _BF, (B, m, d), "tail_x"), (tail_gate, _BF, (B, m, d), "tail_gate"))
    if cache.codes.device != dev:
        raise ValueError(f"cache: must be on {dev}")
    plan.check(dev, B)
    with _on(dev):
        _check(_lib.kv_page_compress(m, x.data_ptr(), gate.data_ptr(), n, row_start.data_ptr(), ctx_len.data_ptr(), B,
                                     pos_bias.data_ptr(), plan.row_start.data_ptr(), plan.row_req.data_ptr(),
                                     plan.row_pos.data_ptr(), plan.slot.data_ptr(), plan.slot.shape[0],
                                     tail_x.data_ptr(), tail_gate.data_ptr(), cache.c_layout, cache.c_struct,
                                     cache.B * cache.capacity, _entry_extras(extras, cache.layout, dev),
                                     _st(dev, stream)), "kv_page_compress")


def paged_attn_workspace_size(n_rows, B, H, layout, max_new, max_entries, W, n_first=0) -> int:
    """Bytes of ws on the current device for paged_attn_chunk (max_entries =
    entry table width x page size, n_first = 0) and paged_attn_window
    (max_entries = 0)."""
    return int(_lib.paged_attn_workspace_size(n_rows, B, H, _layout(layout), max_new or 0, max_entries, W, n_first))


@functools.lru_cache(maxsize=256)
def _ws_bytes(dev, N, B, H, layout, max_new, max_entries, W, n_first):
    with _on(dev):
        return int(_lib.paged_attn_workspace_size(N, B, H, _layout(layout), max_new, max_entries, W, n_first))


def _attn_extras(extras, H, layout, dev):
    if extras is None:
        return None
    for t, shape, n in ((extras.q_norm_w, (layout[0],), "q_norm_w"), (extras.sink, (H,), "sink"),
                        (extras.inv_freq, (layout[1] // 2,), "inv_freq")):
        if t is not None and not _ok(t, _FLOAT, shape, dev):
            _want(dev, (t, _FLOAT, shape, n))
    return ctypes.byref(extras.c_struct())


def _attn(q, row_start, ctx_len, pages, token_table, W, scale, m, cache, entry_table, n_first, max_new, out, ws, stream,
          extras):
    dev = _device(q, "q")
    N, H, d = q.shape
    layout = LAYOUT_512 if d == 512 else LAYOUT_128        # (another d fails the check of q's shape)
    B = ctx_len.shape[0]
    d = layout[0]
    np_, ps, width = pages.shape[0], pages.shape[-2], token_table.shape[-1]
    if not (_ok(q, _BF, (N, H, d), dev) and _ok(row_start, _INT, (B + 1,), dev) and _ok(ctx_len, _INT, (B,), dev)
            and _ok(pages, _BF, (np_, ps, d), dev) and _ok(token_table, _INT, (B, width), dev)):
        _want(dev, (q, _BF, (N, H, d), "q"), (row_start, _INT, (B + 1,), "row_start"), (ctx_len, _INT, (B,), "ctx_len"),
              (pages, _BF, (None, None, d), "pages"), (token_table, _INT, (B, None), "token_table"))
    max_entries = 0
    if cache is not None:
        if cache.layout[0] != d:
            raise ValueError("cache: its layout does not match q")
        if cache.codes.device != dev:
            raise ValueError(f"cache: must be on {dev}")
        e_width = entry_table.shape[-1]
        if not _ok(entry_table, _INT, (B, e_width), dev):
            _want(dev, (entry_table, _INT, (B, None), "entry_table"))
        max_entries = e_width * cache.capacity
    max_new = int(max_new or 0)
    lay = _LAYOUT[layout]
    ex = _attn_extras(extras, H, layout, dev)
    with _on(dev):
        need = _ws_bytes(dev, N, B, H, layout, max_new, max_entries, W, n_first)
        # what is allocated here belongs to the stream that writes it
        if stream is None:
            if out is None:
                out = torch.empty_like(q)
            if need and ws is None:
                ws = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            with torch.cuda.stream(stream):
                if out is None:
                    out = torch.empty_like(q)
                if need and ws is None:
                    ws = torch.empty(need, dtype=torch.uint8, device=dev)
        if not _ok(out, _BF, (N, H, d), dev):
            _want(dev, (out, _BF, (N, H, d), "out"))
        wp, wn = None, 0
        if ws is not None:
            wn = ws.shape[0]
            if not _ok(ws, torch.uint8, (wn,), dev):
                _want(dev, (ws, torch.uint8, (None,), "ws"))
            wp = ws.data_ptr()
        tmap = PageMapStruct(token_table.data_ptr(), width, ps, np_)
        if cache is not None:
            emap = PageMapStruct(entry_table.data_ptr(), e_width, cache.capacity, cache.B)
            _check(_lib.paged_attn_chunk(q.data_ptr(), N, H, B, row_start.data_ptr(), ctx_len.data_ptr(), max_new, m, lay,
                                         cache.c_struct, emap, pages.data_ptr(), tmap, W, scale, ex, out.data_ptr(), wp,
                                         wn, _st(dev, stream)), "paged_attn_chunk")
        else:
            _check(_lib.paged_attn_window(q.data_ptr(), N, H, B, row_start.data_ptr(), ctx_len.data_ptr(), max_new, lay,
                                          pages.data_ptr(), tmap, W, n_first, scale, ex, out.data_ptr(), wp, wn,
                                          _st(dev, stream)), "paged_attn_window")
    return out


def paged_attn_chunk(q, row_start, ctx_len, m: int, cache: KVCache, entry_table, pages, token_table, W: int,
                     softmax_scale: float, max_new=None, out=None, ws=None, stream=None, extras=None):
    """Attention of each request's new tokens over its paged cache: q [n][H][d]
    bf16 (request b's rows row_start[b] ..., at positions ctx_len[b] ...);
    cache + entry_table int32 [B][*]: entries of m tokens in pages; pages bf16
    [pages][page_size][d] + token_table int32 [B][*]: raw tokens in pages, the
    last W of which each query sees.  max_new: a host bound of a request's new
    tokens (1 for a decode step).  Returns out [n][H][d] bf16 (rows past the
    last request's are not written)."""
    return _attn(q, row_start, ctx_len, pages, token_table, W, softmax_scale, m, cache, entry_table, 0, max_new, out, ws,
                 stream, extras)


def paged_attn_window(q, row_start, ctx_len, pages, token_table, W: int, n_first: int, softmax_scale: float,
                      max_new=None, out=None, ws=None, stream=None, extras=None):
    """Attention of each request's new tokens over a sliding window of its paged
    tokens and its first n_first tokens, which stay visible (window-only
    layers); arguments as paged_attn_chunk."""
    return _attn(q, row_start, ctx_len, pages, token_table, W, softmax_scale, 0, None, None, n_first, max_new, out, ws,
                 stream, extras)
