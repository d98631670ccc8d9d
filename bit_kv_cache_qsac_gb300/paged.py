"""Binding of the paged cache (include/qwm_paged.h): many sequences in one pool of pages.

As in the rest of the package the functions mirror the C ABI and only marshal arguments.  Packed
activations are bf16 CUDA tensors of shape [heads, rows, 128] with contiguous channels and otherwise any
strides (a projection's token-major output is passed as a permuted view).  Everything must live on the
context's device; the work is issued on `stream`, or on that device's current stream.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass

import torch

from . import _check, _lib
from .window import _BF16, _R, _S, _array, _rows, _stream_of, qwm_rope_spec, qwm_strides

_P = C.c_void_p
_D, _GROUP = 128, 32
_NO_WINDOW = 1 << 31


class qwm_page_table(C.Structure):
    _fields_ = [("page", C.c_int32), ("batch", C.c_int32), ("width", C.c_int32), ("pages", C.c_int32),
                ("table", _P), ("length", _P), ("free_list", _P), ("free_count", _P)]


class qwm_page_pool(C.Structure):
    _fields_ = [("bits", C.c_int32), ("page", C.c_int32), ("pages", C.c_int32), ("kv_heads", C.c_int32),
                ("k_codes", _P), ("v_codes", _P), ("k_step", _P), ("v_step", _P)]


_T, _O = C.POINTER(qwm_page_table), C.POINTER(qwm_page_pool)
_lib.qwm_norm_rope.argtypes = [_P, _R, _P, _S, C.c_int32, C.c_int32, C.c_int64, _P, _P, _P, _P, C.c_int32, C.c_float, _P, _S,
                               _P]
_lib.qwm_pages_reset.argtypes = [_P, _T, _P]
_lib.qwm_pages_update.argtypes = [_P, _T, _P, _P, C.c_int64, _P, _P, _P, _P, _P]
_lib.qwm_paged_write.argtypes = [_P, _O, _P, _S, _P, _S, C.c_int64, _P, _R, _P, _P, C.c_int32, _P, C.c_int32, C.c_float, _P]
_lib.qwm_paged_read.argtypes = [_P, _O, _P, C.c_int64, _P, _P, _P]
_lib.qwm_paged_attend.argtypes = [_P, _O, _T, _P, _S, C.c_int64, _P, _P, C.c_int64, C.c_int64, C.c_int64, C.c_int64, C.c_float,
                                  _P, _S, C.c_int32, _P, C.c_int32, _P, C.c_size_t, _P]
_lib.qwm_paged_attend_workspace.argtypes = [_P, _O, C.c_int64]
_lib.qwm_paged_attend_workspace.restype = C.c_size_t


@dataclass
class PageTable:
    """Device tensors of a page table, mirroring qwm_page_table: which pages each sequence holds, how many
    tokens it has, and the stack of free pages."""
    page: int
    table: torch.Tensor        # int32 [batch, width]
    length: torch.Tensor       # int64 [batch]
    free: torch.Tensor         # int32 [pages]
    free_count: torch.Tensor   # int32 [1]

    @staticmethod
    def empty(batch: int, width: int, page: int, pages: int, device=None) -> "PageTable":
        """No sequence has tokens and every page is free, page 0 on top; `width`: pages a sequence may
        hold."""
        dev = device or torch.device("cuda", torch.cuda.current_device())
        return PageTable(page, torch.full((batch, width), -1, dtype=torch.int32, device=dev),
                         torch.zeros(batch, dtype=torch.int64, device=dev),
                         torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=dev),
                         torch.full((1,), pages, dtype=torch.int32, device=dev))

    @property
    def batch(self) -> int:
        return self.table.shape[0]

    def struct(self, ctx) -> qwm_page_table:
        b, width = self.table.shape
        pages = self.free.shape[0]
        return qwm_page_table(self.page, b, width, pages, _array(ctx, self.table, "table", torch.int32, (b, width)),
                              _array(ctx, self.length, "length", torch.int64, (b,)),
                              _array(ctx, self.free, "free", torch.int32, (pages,)),
                              _array(ctx, self.free_count, "free_count", torch.int32, (1,)))


@dataclass
class PagePool:
    """Device tensors of one layer's pages, mirroring qwm_page_pool: codes and steps as in Window, slot s in
    page s // page, place s % page."""
    bits: int                # 8 or 4
    k_codes: torch.Tensor    # uint8 [pages, kv_heads, page, 128 * bits / 8]
    k_step: torch.Tensor     # uint8 [pages, kv_heads, page, 4]
    v_codes: torch.Tensor
    v_step: torch.Tensor

    @staticmethod
    def empty(bits: int, page: int, pages: int, kv_heads: int, device=None) -> "PagePool":
        if bits not in (8, 4):
            raise ValueError(f"bits: expected 8 or 4, got {bits}")
        dev = device or torch.device("cuda", torch.cuda.current_device())
        make = lambda w: torch.zeros(pages, kv_heads, page, w, dtype=torch.uint8, device=dev)
        return PagePool(bits, make(_D * bits // 8), make(_D // _GROUP), make(_D * bits // 8), make(_D // _GROUP))

    @property
    def page(self) -> int:
        return self.k_codes.shape[2]

    @property
    def kv_heads(self) -> int:
        return self.k_codes.shape[1]

    def nbytes(self) -> int:
        return sum(t.numel() for t in (self.k_codes, self.k_step, self.v_codes, self.v_step))

    def struct(self, ctx) -> qwm_page_pool:
        if self.bits not in (8, 4):
            raise ValueError(f"bits: expected 8 or 4, got {self.bits}")
        pages, h, page = self.k_codes.shape[:3]
        codes, step, u8 = (pages, h, page, _D * self.bits // 8), (pages, h, page, _D // _GROUP), torch.uint8
        return qwm_page_pool(self.bits, page, pages, h,
                             _array(ctx, self.k_codes, "pool k_codes", u8, codes), _array(ctx, self.v_codes, "pool v_codes", u8, codes),
                             _array(ctx, self.k_step, "pool k_step", u8, step), _array(ctx, self.v_step, "pool v_step", u8, step))


def _packed(ctx, t, name: str, shape, dtypes):
    """Pointer and strides of a packed activation."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise TypeError(f"{name}: expected a tensor [heads][rows][{_D}]")
    return _rows(ctx, t[None], name, (1, *shape), dtypes)


def _weight(ctx, weight, heads: int):
    """Pointer of a norm's weights and whether each head has its own."""
    if weight is None:
        return None, 0
    per_head = isinstance(weight, torch.Tensor) and weight.dim() == 2
    return _array(ctx, weight, "weight", torch.float32, (heads, _D) if per_head else (_D,)), int(per_head)


def qwm_norm_rope(ctx, spec: qwm_rope_spec | None, x, weight, eps: float, out, start=None, at=None, pos=None,
                  stream=None) -> None:
    """out = x [batch, heads, n, 128] divided by the root of each row's mean square, times weight (fp32 [128],
    [heads, 128] or None), then turned by `spec` (or not) at positions start[b] + i, or at[b, i] (int64); out
    may be x.  Tokens at negative positions are left as they were."""
    b, h, n, _ = x.shape
    xp, xs = _rows(ctx, x, "x", (b, h, n, _D), _BF16)
    op, os_ = _rows(ctx, out, "out", (b, h, n, _D), _BF16)
    wp, per_head = _weight(ctx, weight, h)
    _check(_lib.qwm_norm_rope(ctx.handle, C.byref(spec) if spec is not None else None, xp, C.byref(xs), b, h, n,
                              _array(ctx, start, "start", torch.int64, (b,)), _array(ctx, at, "at", torch.int64, (b, n)),
                              _array(ctx, pos, "pos", torch.int32, (b, n, 3)), wp, per_head, float(eps), op, C.byref(os_),
                              _stream_of(ctx, stream)), "qwm_norm_rope")


def qwm_pages_reset(ctx, tab: PageTable, stream=None) -> None:
    """No sequence has tokens and every page is free."""
    t = tab.struct(ctx)
    _check(_lib.qwm_pages_reset(ctx.handle, C.byref(t), _stream_of(ctx, stream)), "qwm_pages_reset")


def qwm_pages_update(ctx, tab: PageTable, first=None, granted=None, slot=None, at=None, count=None, keep=None,
                     stream=None) -> None:
    """Shorten sequences to keep [batch] (int64) tokens, then append count [batch] (int32) new ones: first and
    granted (int32 [batch]), slot and at (int64 [rows]) say where each sequence's rows of the packed batch
    are, how many it was given (its count or 0), and every row's slot and position (-1: padding)."""
    t = tab.struct(ctx)
    b = (tab.batch,)
    n = slot.shape[0] if slot is not None else 0
    _check(_lib.qwm_pages_update(ctx.handle, C.byref(t), _array(ctx, keep, "keep", torch.int64, b),
                                 _array(ctx, count, "count", torch.int32, b), n, _array(ctx, first, "first", torch.int32, b),
                                 _array(ctx, granted, "granted", torch.int32, b), _array(ctx, slot, "slot", torch.int64, (n,)),
                                 _array(ctx, at, "at", torch.int64, (n,)), _stream_of(ctx, stream)), "qwm_pages_update")


def qwm_paged_write(ctx, pool: PagePool, k, v, slot, at=None, rope: qwm_rope_spec | None = None, pos=None, norm: bool = False,
                    weight=None, eps: float = 1e-6, stream=None) -> None:
    """Keys and Values [kv_heads, n, 128] into slot [n] (int64), the Keys normed first (norm, or a weight given)
    and turned by `rope` at positions at [n] (int64)."""
    p = pool.struct(ctx)
    shape = (p.kv_heads, k.shape[1], _D)
    n = shape[1]
    kp, ks = _packed(ctx, k, "k", shape, _BF16)
    vp, vs = _packed(ctx, v, "v", shape, _BF16)
    wp, per_head = _weight(ctx, weight, p.kv_heads)
    _check(_lib.qwm_paged_write(ctx.handle, C.byref(p), kp, C.byref(ks), vp, C.byref(vs), n,
                                _array(ctx, slot, "slot", torch.int64, (n,)), C.byref(rope) if rope is not None else None,
                                _array(ctx, at, "at", torch.int64, (n,)), _array(ctx, pos, "pos", torch.int32, (n, 3)),
                                int(norm or weight is not None), wp, per_head, float(eps), _stream_of(ctx, stream)),
           "qwm_paged_write")


def qwm_paged_read(ctx, pool: PagePool, slot, k_hat, v_hat, stream=None) -> None:
    """What the slots [n] stand for, in bf16 [kv_heads, n, 128] (either of k_hat and v_hat may be None); negative
    slots read as 0."""
    p = pool.struct(ctx)
    n = slot.shape[0]
    ptr = []
    for t, name in ((k_hat, "k_hat"), (v_hat, "v_hat")):
        if t is not None and t.dtype not in _BF16:
            raise TypeError(f"{name}: expected bfloat16, got {t.dtype}")
        ptr.append(_array(ctx, t, name, t.dtype, (p.kv_heads, n, _D)) if t is not None else None)
    _check(_lib.qwm_paged_read(ctx.handle, C.byref(p), _array(ctx, slot, "slot", torch.int64, (n,)), n, *ptr,
                               _stream_of(ctx, stream)), "qwm_paged_read")


def qwm_paged_attend_workspace(ctx, pool: PagePool, max_count: int) -> int:
    """Bytes of workspace for calls of up to max_count new tokens a sequence."""
    p = pool.struct(ctx)
    return _lib.qwm_paged_attend_workspace(ctx.handle, C.byref(p), max_count)


def qwm_paged_attend(ctx, pool: PagePool, tab: PageTable, q, first, count, softmax_scale: float, out, lse=None,
                     merge: bool = False, tpf: int = 1, frames: int | None = None, sink: int = 0, max_count: int | None = None,
                     ws=None, stream=None) -> None:
    """Attention of packed Queries [H, n, 128], rows first[b] .. of sequence b its newest count[b] tokens, over its
    pages: the tokens of the last `frames` frames of `tpf` tokens (None: all) and the first `sink`.  out: bf16 or
    fp32; lse: fp32 [H, n] or None; merge: out (fp32) and lse hold a result over other keys and become the
    result over both.  max_count: the largest count, or more (None: n).  ws: a uint8 workspace tensor, or None to
    allocate one (on the call's stream)."""
    p, t = pool.struct(ctx), tab.struct(ctx)
    H, n = ctx.heads, q.shape[1]
    shape = (H, n, _D)
    qp, qs = _packed(ctx, q, "q", shape, _BF16)
    op, os_ = _packed(ctx, out, "out", shape, _BF16 + (torch.float32,))
    most = n if max_count is None else int(max_count)
    if ws is None:
        key = (p.bits, p.kv_heads, most)
        need = ctx.paged_workspace.get(key)
        if need is None:
            if len(ctx.paged_workspace) > 1000:
                ctx.paged_workspace.clear()
            need = ctx.paged_workspace[key] = _lib.qwm_paged_attend_workspace(ctx.handle, C.byref(p), most)
        if stream is None:
            ws = torch.empty(need, dtype=torch.uint8, device=ctx.device)
        else:
            s = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), ctx.device)
            with torch.cuda.stream(s):
                ws = torch.empty(need, dtype=torch.uint8, device=ctx.device)
    b = (t.batch,)
    _check(_lib.qwm_paged_attend(ctx.handle, C.byref(p), C.byref(t), qp, C.byref(qs), n, _array(ctx, first, "first", torch.int32, b),
                                 _array(ctx, count, "count", torch.int32, b), most, tpf, _NO_WINDOW if frames is None else frames,
                                 sink, float(softmax_scale), op, C.byref(os_), int(out.dtype == torch.float32),
                                 _array(ctx, lse, "lse", torch.float32, shape[:2]), int(bool(merge)),
                                 _array(ctx, ws, "ws", torch.uint8, (ws.numel(),)), ws.numel(), _stream_of(ctx, stream)),
           "qwm_paged_attend")
