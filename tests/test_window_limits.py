"""Host-side limits of the recent window (no GPU)."""
import ctypes as C
import os
import subprocess
import sys

import pytest

import window_ref as ref


@pytest.fixture(scope="module")
def qwm():
    import __graft_entry__
    __graft_entry__.build_library()
    import bit_kv_cache_qsac_gb300 as q
    return q


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("theta", [1.0, 2.0, 256.0, 1e4, 123456.789, 5e5, 1e300, (1e4, 1e3, 50.0)])
@pytest.mark.parametrize("dims", [(128, 0, 0), (44, 42, 42), (2, 4, 30)])
def test_plan_turns_are_rounded_once(qwm, dims, theta, shared, inverse):
    """Each entry is the exact part of a turn to half a unit of 2^-64 (2^-20 of a unit for the arithmetic of
    some 100 bits): positions multiply what is left."""
    spec = qwm.RopeSpec(dims, theta=theta, shared_freq=shared, inverse=inverse)
    exact = ref.exact_turns(dims, theta if isinstance(theta, tuple) else (theta,) * 3, shared)
    for i, t in enumerate(exact):
        got = spec.turn[i] if not inverse else -spec.turn[i] % 2 ** 64
        assert abs(got * 2 ** 136 - t) <= 2 ** 135 + 2 ** 116, (i, got, t / 2 ** 136)


def test_long_calls_are_split(qwm):
    """No part of a call takes more than 2^18 keys (here without a device: a context of no SMs, which plans no
    parts for speed)."""
    ctx = (C.c_char * 4096)()
    cfg = qwm.qwm_config(8, 128, 256, 64, 4, 8, 2, 10, 0)
    C.memmove(ctx, C.byref(cfg), C.sizeof(cfg))
    lib = qwm.raw_library()
    for sink, ring, nq, frames, parts in ((0, 1 << 18, 1, 1 << 30, 0), (1, 1 << 18, 1, 1 << 30, 2), (0, 1 << 20, 40, 1 << 30, 4),
                                          (0, (1 << 20) + 1, 600, 1 << 30, 5), (0, 1 << 30, 1, 1 << 30, 4096), (0, 1 << 30, 600, 1 << 30, 4096),
                                          (0, 1 << 30, 1, 1 << 17, 0), (5, 1 << 30, 600, (1 << 18) - 1024, 0)):
        w = qwm.qwm_window(4, 2, 4, 0, sink, ring)
        need = lib.qwm_window_attend_workspace(ctx, w, nq, 1, frames)
        assert need == 2 * 8 * nq * parts * 129 * 4, (sink, ring, nq, frames, need / (2 * 8 * nq * 129 * 4))


def test_softmax_scale_range(qwm):
    """A scale whose product with log2(e) and the 4-bit unit is infinite would make 0 logits NaN."""
    ctx, ok = (C.c_char * 4096)(), 0x7f00000000
    cfg = qwm.qwm_config(8, 128, 256, 64, 4, 8, 2, 10, 0)
    C.memmove(ctx, C.byref(cfg), C.sizeof(cfg))
    st = qwm.qwm_strides(8 * 128 * 4, 128 * 4, 128)
    for bits in (8, 4):
        w = qwm.qwm_window(bits, 2, 4, 0, 4, 100, ok, ok, ok, ok)
        for scale, nq, want in ((2.0 ** 123, 0, qwm.QWM_OK), (2.0 ** 123 * (1 + 2.0 ** -23), 0, qwm.QWM_ERR_ARG), (3.4e38, 0, qwm.QWM_ERR_ARG),
                                (3.4e38, 4, qwm.QWM_ERR_ARG)):
            assert qwm.raw_library().qwm_window_attend(ctx, w, ok, st, nq, ok, ok, None, 1, 8, scale, ok, st, 0, None, 0, None, 0, None) == want


def test_import_without_torchs_private_stream_handle(qwm):
    """The package loads with a torch that lacks the call behind torch.cuda.current_stream."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import torch; torch._C.__dict__.get('_cuda_getCurrentRawStream') and delattr(torch._C, '_cuda_getCurrentRawStream'); "
            "import bit_kv_cache_qsac_gb300.window as w; assert callable(w._current_stream)")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-500:]
