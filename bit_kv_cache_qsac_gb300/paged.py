"""Binding of the paged cache (include/qwm_paged.h): many sequences in one pool of pages.

As in the rest of the package the functions mirror the C ABI and only marshal arguments.  Packed
activations are bf16 CUDA tensors of shape [heads, rows, 128] with contiguous channels and otherwise any
strides (a projection's token-major output is passed as a permuted view).  Everything must live on the
context's device; the work is issued on `stream`, or on that device's current stream.
"""
from __future__ import annotations

import ctypes as C
import struct
from dataclasses import dataclass
from types import SimpleNamespace

import torch

from . import LIB_PATH, _check, _lib
from .window import _BF16, _R, _S, _refuse, _stream_of, qwm_rope_spec

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
_I32, _I64, _F32 = C.c_int32, C.c_int64, C.c_float


def _declare(lib, rope, strides, table, pool) -> None:
    lib.qwm_norm_rope.argtypes = [_P, rope, _P, strides, _I32, _I32, _I64, _P, _P, _P, _P, _I32, _F32, _P, strides, _P]
    lib.qwm_pages_reset.argtypes = [_P, table, _P]
    lib.qwm_pages_update.argtypes = [_P, table, _P, _P, _I64, _P, _P, _P, _P, _P]
    lib.qwm_paged_write.argtypes = [_P, pool, _P, strides, _P, strides, _I64, _P, rope, _P, _P, _I32, _P, _I32, _F32, _P]
    lib.qwm_paged_read.argtypes = [_P, pool, _P, _I64, _P, _P, _P]
    lib.qwm_paged_attend.argtypes = [_P, pool, table, _P, strides, _I64, _P, _P, _I64, _I64, _I64, _I64, _F32, _P, strides, _I32, _P,
                                     _I32, _P, C.c_size_t, _P]
    lib.qwm_paged_attend_workspace.argtypes = [_P, pool, _I64]
    lib.qwm_paged_attend_workspace.restype = C.c_size_t


_declare(_lib, _R, _S, _T, _O)
# The same functions for this module's own calls, which pass structures as packed bytes: a ctypes structure
# takes four times as long to make, and a call of a few microseconds' work passes five of them.
_fast = C.CDLL(LIB_PATH)
_declare(_fast, _P, _P, _P, _P)
_pack_table = _pack_pool = struct.Struct("iiiiPPPP").pack   # qwm_page_table, qwm_page_pool
_pack_strides = struct.Struct("qqq").pack                   # qwm_strides
_U8, _BF = torch.uint8, torch.bfloat16


def _wrong(dev, t, name: str, dtypes, shape):
    _refuse(SimpleNamespace(device=dev), t, name, dtypes, shape)


def _dense(dev, t, name: str, dtype, shape):
    """Pointer of a dense device array (or None)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        _wrong(dev, t, name, (dtype,), shape)
    return t.data_ptr()


def _packed(dev, t, name: str, shape, dtypes=_BF16):
    """Pointer and strides of a packed activation [heads, rows, 128]."""
    if not isinstance(t, torch.Tensor) or (t.dtype is not _BF and t.dtype not in dtypes) or t.shape != shape or t.device != dev:
        _wrong(dev, t, name, dtypes, shape)
    h, n, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: channels must be contiguous")
    return t.data_ptr(), _pack_strides(0, h if shape[0] > 1 else 0, n if shape[1] > 1 else 0)


def _rows4(dev, t, name: str, shape):
    """Pointer and strides of an activation [batch, heads, tokens, 128]."""
    if not isinstance(t, torch.Tensor) or (t.dtype is not _BF and t.dtype not in _BF16) or t.shape != shape or t.device != dev:
        _wrong(dev, t, name, _BF16, shape)
    b, h, n, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: channels must be contiguous")
    return t.data_ptr(), _pack_strides(b if shape[0] > 1 else 0, h if shape[1] > 1 else 0, n if shape[2] > 1 else 0)


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

    def packed(self, dev) -> bytes:
        """The qwm_page_table, its tensors looked at."""
        b, width = self.table.shape
        pages = self.free.shape[0]
        return _pack_table(self.page, b, width, pages, _dense(dev, self.table, "table", torch.int32, (b, width)),
                           _dense(dev, self.length, "length", torch.int64, (b,)), _dense(dev, self.free, "free", torch.int32, (pages,)),
                           _dense(dev, self.free_count, "free_count", torch.int32, (1,)))


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

    def packed(self, dev) -> bytes:
        """The qwm_page_pool, its tensors looked at."""
        bits = self.bits
        if bits not in (8, 4):
            raise ValueError(f"bits: expected 8 or 4, got {bits}")
        pages, h, page = self.k_codes.shape[:3]
        codes, step = (pages, h, page, _D * bits // 8), (pages, h, page, _D // _GROUP)
        return _pack_pool(bits, page, pages, h, _dense(dev, self.k_codes, "pool k_codes", _U8, codes),
                          _dense(dev, self.v_codes, "pool v_codes", _U8, codes), _dense(dev, self.k_step, "pool k_step", _U8, step),
                          _dense(dev, self.v_step, "pool v_step", _U8, step))


def _weight(dev, weight, heads: int):
    """Pointer of a norm's weights and whether each head has its own."""
    if weight is None:
        return None, 0
    per_head = isinstance(weight, torch.Tensor) and weight.dim() == 2
    return _dense(dev, weight, "weight", torch.float32, (heads, _D) if per_head else (_D,)), int(per_head)


def _spec(spec):
    return C.addressof(spec) if spec is not None else None


def qwm_norm_rope(ctx, spec: qwm_rope_spec | None, x, weight, eps: float, out, start=None, at=None, pos=None,
                  stream=None) -> None:
    """out = x [batch, heads, n, 128] divided by the root of each row's mean square, times weight (fp32 [128],
    [heads, 128] or None), then turned by `spec` (or not) at positions start[b] + i, or at[b, i] (int64); out
    may be x.  Tokens at negative positions are left as they were."""
    dev, (b, h, n, _) = ctx.device, x.shape
    xp, xs = _rows4(dev, x, "x", (b, h, n, _D))
    op, os_ = _rows4(dev, out, "out", (b, h, n, _D))
    wp, per_head = _weight(dev, weight, h)
    _check(_fast.qwm_norm_rope(ctx.handle, _spec(spec), xp, xs, b, h, n, _dense(dev, start, "start", torch.int64, (b,)),
                               _dense(dev, at, "at", torch.int64, (b, n)), _dense(dev, pos, "pos", torch.int32, (b, n, 3)), wp, per_head,
                               eps, op, os_, _stream_of(ctx, stream)), "qwm_norm_rope")


def qwm_pages_reset(ctx, tab: PageTable, stream=None) -> None:
    """No sequence has tokens and every page is free."""
    _check(_fast.qwm_pages_reset(ctx.handle, tab.packed(ctx.device), _stream_of(ctx, stream)), "qwm_pages_reset")


def qwm_pages_update(ctx, tab: PageTable, first=None, granted=None, slot=None, at=None, count=None, keep=None,
                     stream=None) -> None:
    """Shorten sequences to keep [batch] (int64) tokens, then append count [batch] (int32) new ones: first and
    granted (int32 [batch]), slot and at (int64 [rows]) say where each sequence's rows of the packed batch
    are, how many it was given (its count or 0), and every row's slot and position (-1: padding)."""
    dev = ctx.device
    b, n = (tab.table.shape[0],), slot.shape[0] if slot is not None else 0
    _check(_fast.qwm_pages_update(ctx.handle, tab.packed(dev), _dense(dev, keep, "keep", torch.int64, b),
                                  _dense(dev, count, "count", torch.int32, b), n, _dense(dev, first, "first", torch.int32, b),
                                  _dense(dev, granted, "granted", torch.int32, b), _dense(dev, slot, "slot", torch.int64, (n,)),
                                  _dense(dev, at, "at", torch.int64, (n,)), _stream_of(ctx, stream)), "qwm_pages_update")


def qwm_paged_write(ctx, pool: PagePool, k, v, slot, at=None, rope: qwm_rope_spec | None = None, pos=None, norm: bool = False,
                    weight=None, eps: float = 1e-6, stream=None) -> None:
    """Keys and Values [kv_heads, n, 128] into slot [n] (int64), the Keys normed first (norm, or a weight given)
    and turned by `rope` at positions at [n] (int64)."""
    dev, p = ctx.device, pool.packed(ctx.device)
    h, n = pool.k_codes.shape[1], k.shape[1]
    kp, ks = _packed(dev, k, "k", (h, n, _D))
    vp, vs = _packed(dev, v, "v", (h, n, _D))
    wp, per_head = _weight(dev, weight, h)
    _check(_fast.qwm_paged_write(ctx.handle, p, kp, ks, vp, vs, n, _dense(dev, slot, "slot", torch.int64, (n,)), _spec(rope),
                                 _dense(dev, at, "at", torch.int64, (n,)), _dense(dev, pos, "pos", torch.int32, (n, 3)),
                                 int(norm or weight is not None), wp, per_head, eps, _stream_of(ctx, stream)), "qwm_paged_write")


def qwm_paged_read(ctx, pool: PagePool, slot, k_hat, v_hat, stream=None) -> None:
    """What the slots [n] stand for, in bf16 [kv_heads, n, 128] (either of k_hat and v_hat may be None); negative
    slots read as 0."""
    dev, p = ctx.device, pool.packed(ctx.device)
    n, h = slot.shape[0], pool.k_codes.shape[1]
    ptr = []
    for t, name in ((k_hat, "k_hat"), (v_hat, "v_hat")):
        if t is not None and t.dtype not in _BF16:
            raise TypeError(f"{name}: expected bfloat16, got {t.dtype}")
        ptr.append(_dense(dev, t, name, t.dtype, (h, n, _D)) if t is not None else None)
    _check(_fast.qwm_paged_read(ctx.handle, p, _dense(dev, slot, "slot", torch.int64, (n,)), n, *ptr, _stream_of(ctx, stream)),
           "qwm_paged_read")


def qwm_paged_attend_workspace(ctx, pool: PagePool, max_count: int) -> int:
    """Bytes of workspace for calls of up to max_count new tokens a sequence."""
    return _fast.qwm_paged_attend_workspace(ctx.handle, pool.packed(ctx.device), max_count)


_OUT = _BF16 + (torch.float32,)


def qwm_paged_attend(ctx, pool: PagePool, tab: PageTable, q, first, count, softmax_scale: float, out, lse=None,
                     merge: bool = False, tpf: int = 1, frames: int | None = None, sink: int = 0, max_count: int | None = None,
                     ws=None, stream=None) -> None:
    """Attention of packed Queries [H, n, 128], rows first[b] .. of sequence b its newest count[b] tokens, over its
    pages: the tokens of the last `frames` frames of `tpf` tokens (None: all) and the first `sink`.  out: bf16 or
    fp32; lse: fp32 [H, n] or None; merge: out (fp32) and lse hold a result over other keys and become the
    result over both.  max_count: the largest count, or more (None: n): the kernels are chosen by it, and those for long
    prompts cost a step of single tokens 4 to 9 us and 40 MB of workspace where it says that there may be one.
    ws: a uint8 workspace tensor, or None to allocate one (on the call's stream)."""
    dev = ctx.device
    p, t = pool.packed(dev), tab.packed(dev)
    n = q.shape[1]
    shape, b = (ctx.heads, n, _D), (tab.table.shape[0],)
    qp, qs = _packed(dev, q, "q", shape)
    op, os_ = _packed(dev, out, "out", shape, _OUT)
    most = n if max_count is None else int(max_count)
    if ws is None:
        key = (pool.bits, pool.k_codes.shape[1], most)   # all that the size depends on, beside the context
        need = ctx.paged_workspace.get(key)
        if need is None:
            need = _fast.qwm_paged_attend_workspace(ctx.handle, p, most)
            if need:   # (0: a call that will be refused, for what the key does not hold)
                if len(ctx.paged_workspace) > 1000:
                    ctx.paged_workspace.clear()
                ctx.paged_workspace[key] = need
        if stream is None:
            ws = torch.empty(need, dtype=_U8, device=dev)
        else:
            s = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), dev)
            with torch.cuda.stream(s):
                ws = torch.empty(need, dtype=_U8, device=dev)
    size = ws.numel()
    _check(_fast.qwm_paged_attend(ctx.handle, p, t, qp, qs, n, _dense(dev, first, "first", torch.int32, b),
                                  _dense(dev, count, "count", torch.int32, b), most, tpf, _NO_WINDOW if frames is None else frames, sink,
                                  softmax_scale, op, os_, int(out.dtype is torch.float32),
                                  _dense(dev, lse, "lse", torch.float32, shape[:2]), int(bool(merge)),
                                  _dense(dev, ws, "ws", _U8, (size,)), size, _stream_of(ctx, stream)), "qwm_paged_attend")
