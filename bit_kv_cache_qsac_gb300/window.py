"""Binding of the recent window (include/qwm_window.h): rotary positions, the window cache and the
attention over it.

As in the rest of the package the functions mirror the C ABI and only marshal arguments.  Activations
are bf16 CUDA tensors of shape [batch, heads, tokens, 128] with contiguous channels and otherwise any
strides (a projection's token-major output is passed as a permuted view).  Everything must live on the
context's device; the work is issued on `stream`, or on that device's current stream.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass

import torch

from . import _check, _lib

_P = C.c_void_p
_D, _GROUP = 128, 32

QWM_ROPE_INTERLEAVED, QWM_ROPE_HALF = 0, 1
_PAIRING = {"interleaved": QWM_ROPE_INTERLEAVED, "half": QWM_ROPE_HALF}


class qwm_strides(C.Structure):
    _fields_ = [("batch", C.c_int64), ("head", C.c_int64), ("token", C.c_int64)]


class qwm_rope_spec(C.Structure):
    _fields_ = [("rot", C.c_int32), ("pairing", C.c_int32), ("grid_h", C.c_int32), ("grid_w", C.c_int32),
                ("turn", C.c_uint64 * 64), ("axis", C.c_uint8 * 64)]


class qwm_window(C.Structure):
    _fields_ = [("bits", C.c_int32), ("batch", C.c_int32), ("kv_heads", C.c_int32), ("reserved", C.c_int32),
                ("sink", C.c_int64), ("ring", C.c_int64),
                ("k_codes", _P), ("v_codes", _P), ("k_step", _P), ("v_step", _P)]


_S, _W, _R = C.POINTER(qwm_strides), C.POINTER(qwm_window), C.POINTER(qwm_rope_spec)
_lib.qwm_rope_plan.argtypes = [C.POINTER(C.c_int32), C.POINTER(C.c_double), C.c_int32, C.c_int32, C.c_int32, C.c_int32,
                               C.c_int32, _R]
_lib.qwm_rope.argtypes = [_P, _R, _P, _S, C.c_int32, C.c_int32, C.c_int64, _P, _P, _P, _S, _P]
_lib.qwm_window_bytes.argtypes = [_W, C.POINTER(C.c_size_t), C.POINTER(C.c_size_t)]
_lib.qwm_window_write.argtypes = [_P, _W, _P, _S, _P, _S, C.c_int64, _P, _P, _R, _P, _P]
_lib.qwm_window_read.argtypes = [_P, _W, _P, _P, _P, C.c_int64, _P, _P, _P]
_lib.qwm_window_attend.argtypes = [_P, _W, _P, _S, C.c_int64, _P, _P, _P, C.c_int64, C.c_int64, C.c_float, _P, _S,
                                   C.c_int32, _P, C.c_int32, _P, C.c_size_t, _P]
_lib.qwm_window_attend_workspace.argtypes = [_P, _W, C.c_int64, C.c_int64, C.c_int64]
_lib.qwm_window_attend_workspace.restype = C.c_size_t


def qwm_rope_plan(axis_dim, theta, pairing: int, shared_freq: int, grid_h: int, grid_w: int, inverse: int,
                  out: qwm_rope_spec) -> None:
    """Host: fill a rotation (see RopeSpec)."""
    _check(_lib.qwm_rope_plan((C.c_int32 * 3)(*axis_dim), (C.c_double * 3)(*theta), pairing, shared_freq, grid_h,
                              grid_w, inverse, C.byref(out)), "qwm_rope_plan")


class RopeSpec(qwm_rope_spec):
    """A rotation with three axes (time, height, width).

    dims: channels of the t, y and x sections (even; the channels past their sum pass through); theta: the
    frequencies' base, one number or one per axis; pairing: "interleaved" (channels 2 i, 2 i + 1) or "half"
    (i, i + R / 2); shared_freq: one frequency ladder over all pairs instead of one per axis; grid:
    (height, width) of a frame, from which a token's place follows ((1, 1): one axis); inverse: turn
    back (also the gradient of the rotation)."""

    def __init__(self, dims, theta=10000.0, pairing: str = "interleaved", shared_freq: bool = False, grid=(1, 1),
                 inverse: bool = False):
        super().__init__()
        if pairing not in _PAIRING:
            raise ValueError(f"pairing: expected one of {sorted(_PAIRING)}, got {pairing!r}")
        bases = [float(t) for t in theta] if isinstance(theta, (tuple, list)) else [float(theta)] * 3
        if len(dims) != 3 or len(bases) != 3:
            raise ValueError("dims and theta take one entry per axis (t, y, x)")
        qwm_rope_plan([int(m) for m in dims], bases, _PAIRING[pairing], int(bool(shared_freq)), int(grid[0]), int(grid[1]),
                      int(bool(inverse)), self)


def _refuse(ctx, t, name: str, dtypes, shape) -> None:
    """Raise what is wrong with a tensor (the checks that failed together in the callers)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if t.device != ctx.device:
        raise ValueError(f"{name}: on {t.device}, the context is on {ctx.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: tensor must be contiguous")


def _rows(ctx, t, name: str, shape, dtypes):
    """Pointer and strides of an activation."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.shape != shape or t.device != ctx.device:
        _refuse(ctx, t, name, dtypes, shape)
    b, h, n, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: channels must be contiguous")
    return t.data_ptr(), qwm_strides(b if shape[0] > 1 else 0, h if shape[1] > 1 else 0, n if shape[2] > 1 else 0)


def check_rows(ctx, t, name: str, shape) -> None:
    """Raise unless t is an activation the calls take: shape, 16-bit elements, the context's device, rows
    that start on 16-byte boundaries."""
    at, strides = _rows(ctx, t, name, shape, _BF16)
    if at % 16 or any(s % 8 for s in (strides.batch, strides.head, strides.token)):
        raise ValueError(f"{name}: rows must start on 16-byte boundaries")


def _array(ctx, t, name: str, dtype, shape) -> int | None:
    """Pointer of a dense device array (or None)."""
    if t is None:
        return None
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.device != ctx.device or
            not t.is_contiguous()):
        _refuse(ctx, t, name, (dtype,), shape)
    return t.data_ptr()


# the handle itself, at a tenth of torch.cuda.current_stream's time, where this torch has it
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream_of(ctx, stream) -> int:
    if stream is None:
        return _current_stream(ctx.device.index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)   # 16-bit integers hold the bit patterns


@dataclass
class Window:
    """Device tensors of a window cache, mirroring qwm_window: slots 0 .. sink - 1 keep the first tokens
    of a sequence, token p >= sink lives in slot sink + (p - sink) % ring."""
    bits: int                # 8 or 4
    sink: int
    ring: int
    k_codes: torch.Tensor    # uint8 [batch, kv_heads, sink + ring, 128 * bits / 8]
    k_step: torch.Tensor     # uint8 [batch, kv_heads, sink + ring, 4]
    v_codes: torch.Tensor
    v_step: torch.Tensor

    @staticmethod
    def empty(bits: int, batch: int, kv_heads: int, sink: int, ring: int, device=None) -> "Window":
        """An unwritten cache on `device` (default: the current one)."""
        if bits not in (8, 4):
            raise ValueError(f"bits: expected 8 or 4, got {bits}")
        dev = device or torch.device("cuda", torch.cuda.current_device())
        make = lambda w: torch.zeros(batch, kv_heads, sink + ring, w, dtype=torch.uint8, device=dev)
        return Window(bits, sink, ring, make(_D * bits // 8), make(_D // _GROUP), make(_D * bits // 8), make(_D // _GROUP))

    @property
    def batch(self) -> int:
        return self.k_codes.shape[0]

    @property
    def kv_heads(self) -> int:
        return self.k_codes.shape[1]

    def nbytes(self) -> int:
        return sum(t.numel() for t in (self.k_codes, self.k_step, self.v_codes, self.v_step))

    def struct(self, ctx) -> qwm_window:
        if self.bits not in (8, 4):
            raise ValueError(f"bits: expected 8 or 4, got {self.bits}")
        b, h = self.k_codes.shape[:2]
        lead = (b, h, self.sink + self.ring)
        codes, step = lead + (_D * self.bits // 8,), lead + (_D // _GROUP,)
        u8 = torch.uint8
        return qwm_window(self.bits, b, h, 0, self.sink, self.ring,
                          _array(ctx, self.k_codes, "window k_codes", u8, codes), _array(ctx, self.v_codes, "window v_codes", u8, codes),
                          _array(ctx, self.k_step, "window k_step", u8, step), _array(ctx, self.v_step, "window v_step", u8, step))


def qwm_window_bytes(bits: int, batch: int, kv_heads: int, sink: int, ring: int) -> tuple[int, int]:
    """Host: bytes of one codes array and of one step array."""
    w = qwm_window(bits, batch, kv_heads, 0, sink, ring)
    codes, step = C.c_size_t(), C.c_size_t()
    _check(_lib.qwm_window_bytes(C.byref(w), C.byref(codes), C.byref(step)), "qwm_window_bytes")
    return codes.value, step.value


def qwm_rope(ctx, spec: qwm_rope_spec, x, start, out, pos=None, stream=None) -> None:
    """out = x turned by its positions start[b] + i (or by pos int32 [batch, n, 3]); out may be x."""
    b, h, n, _ = x.shape
    xp, xs = _rows(ctx, x, "x", (b, h, n, _D), _BF16)
    op, os_ = _rows(ctx, out, "out", (b, h, n, _D), _BF16)
    _check(_lib.qwm_rope(ctx.handle, C.byref(spec), xp, C.byref(xs), b, h, n, _array(ctx, start, "start", torch.int64, (b,)),
                         _array(ctx, pos, "pos", torch.int32, (b, n, 3)), op, C.byref(os_), _stream_of(ctx, stream)),
           "qwm_rope")


def qwm_window_write(ctx, win: Window, k, v, start, count=None, rope: qwm_rope_spec | None = None, pos=None,
                     stream=None) -> None:
    """Append tokens start[b] .. start[b] + count[b] - 1 (count: n without it), the Keys turned by `rope`."""
    w = win.struct(ctx)
    n = k.shape[2]
    shape = (w.batch, w.kv_heads, n, _D)
    kp, ks = _rows(ctx, k, "k", shape, _BF16)
    vp, vs = _rows(ctx, v, "v", shape, _BF16)
    _check(_lib.qwm_window_write(ctx.handle, C.byref(w), kp, C.byref(ks), vp, C.byref(vs), n,
                                 _array(ctx, start, "start", torch.int64, (w.batch,)),
                                 _array(ctx, count, "count", torch.int32, (w.batch,)),
                                 C.byref(rope) if rope is not None else None,
                                 _array(ctx, pos, "pos", torch.int32, (w.batch, n, 3)), _stream_of(ctx, stream)),
           "qwm_window_write")


def qwm_window_read(ctx, win: Window, start, length, k_hat, v_hat, count=None, stream=None) -> None:
    """Tokens start[b] .. of sequences of length[b] tokens in bf16 [batch, kv_heads, n, 128] (either of
    k_hat and v_hat may be None); tokens the cache does not hold read as 0."""
    w = win.struct(ctx)
    some = k_hat if k_hat is not None else v_hat
    if some is None:
        return
    n = some.shape[2]
    shape = (w.batch, w.kv_heads, n, _D)
    ptr = []
    for t, name in ((k_hat, "k_hat"), (v_hat, "v_hat")):
        if t is not None and t.dtype not in _BF16:
            raise TypeError(f"{name}: expected bfloat16, got {t.dtype}")
        ptr.append(_array(ctx, t, name, t.dtype, shape) if t is not None else None)
    _check(_lib.qwm_window_read(ctx.handle, C.byref(w), _array(ctx, start, "start", torch.int64, (w.batch,)),
                                _array(ctx, length, "length", torch.int64, (w.batch,)),
                                _array(ctx, count, "count", torch.int32, (w.batch,)), n, *ptr, _stream_of(ctx, stream)),
           "qwm_window_read")


def qwm_window_attend_workspace(ctx, win: Window, nq: int, tpf: int, frames: int) -> int:
    """Bytes of workspace qwm_window_attend needs for this shape (0: none)."""
    w = win.struct(ctx)
    return _lib.qwm_window_attend_workspace(ctx.handle, C.byref(w), nq, tpf, frames)


def qwm_window_attend(ctx, win: Window, q, q_start, length, tpf: int, frames: int, softmax_scale: float, out, lse=None,
                      merge: bool = False, q_count=None, ws=None, stream=None) -> None:
    """Attention of Queries [batch, H, nq, 128] at positions q_start[b] + i over the cached tokens: keys of
    the last `frames` frames of `tpf` tokens and of the sinks.  out: bf16 or fp32; lse: fp32 [batch, H, nq]
    or None; merge: out (fp32) and lse hold a result over other keys and become the result over both.
    ws: a uint8 workspace tensor, or None to allocate one (on the call's stream) when one is needed."""
    w = win.struct(ctx)
    nq, H = q.shape[2], ctx.heads
    shape = (w.batch, H, nq, _D)
    qp, qs = _rows(ctx, q, "q", shape, _BF16)
    op, os_ = _rows(ctx, out, "out", shape, _BF16 + (torch.float32,))
    key = (w.batch, w.kv_heads, w.sink, w.ring, nq, tpf, frames)   # all the size depends on, beside the context
    need = ctx.window_workspace.get(key)
    if need is None:
        need = ctx.window_workspace[key] = _lib.qwm_window_attend_workspace(ctx.handle, C.byref(w), nq, tpf, frames)
        if len(ctx.window_workspace) > 1000:
            ctx.window_workspace.clear()
    if need and ws is None:
        if stream is None:
            ws = torch.empty(need, dtype=torch.uint8, device=ctx.device)
        else:
            s = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), ctx.device)
            with torch.cuda.stream(s):
                ws = torch.empty(need, dtype=torch.uint8, device=ctx.device)
    if ws is not None:
        _array(ctx, ws, "ws", torch.uint8, (ws.numel(),))
    _check(_lib.qwm_window_attend(ctx.handle, C.byref(w), qp, C.byref(qs), nq,
                                  _array(ctx, q_start, "q_start", torch.int64, (w.batch,)),
                                  _array(ctx, length, "length", torch.int64, (w.batch,)),
                                  _array(ctx, q_count, "q_count", torch.int32, (w.batch,)), tpf, frames, float(softmax_scale),
                                  op, C.byref(os_), int(out.dtype == torch.float32),
                                  _array(ctx, lse, "lse", torch.float32, shape[:3]), int(bool(merge)),
                                  ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0,
                                  _stream_of(ctx, stream)), "qwm_window_attend")
