"""Host-side checks of the recent window (no GPU): the rotation plan, sizes, and every refusal, which
comes before the first CUDA call."""
import ctypes as C

import numpy as np
import pytest

import window_ref as ref


@pytest.fixture(scope="module")
def qwm():
    import __graft_entry__
    __graft_entry__.build_library()
    import bit_kv_cache_qsac_gb300 as q
    return q


def _ctx(qwm, heads=8):
    """A context that has no device side: enough for calls that are refused (the configuration leads
    the structure)."""
    buf = (C.c_char * 4096)()
    cfg = qwm.qwm_config(heads, 128, 256, 64, 4, 8, 2, 10, 0)
    C.memmove(buf, C.byref(cfg), C.sizeof(cfg))
    return buf


def test_plan_turns_and_axes(qwm):
    for dims, theta, pairing, shared, inverse in (((44, 42, 42), 10000.0, "interleaved", False, False),
                                                  ((32, 16, 16), (10000.0, 100.0, 1.0), "half", False, True),
                                                  ((16, 56, 56), 1e6, "half", True, False), ((0, 0, 0), 2.0, "half", False, False)):
        s = qwm.RopeSpec(dims, theta=theta, pairing=pairing, shared_freq=shared, grid=(3, 5), inverse=inverse)
        base = theta if isinstance(theta, tuple) else (theta,) * 3
        assert (s.rot, s.grid_h, s.grid_w) == (sum(dims), 3, 5)
        i = 0
        for a in range(3):
            for j in range(dims[a] // 2):
                rate = base[a] ** (-(2.0 * i / sum(dims) if shared else 2.0 * j / dims[a]))
                t = s.turn[i] if not inverse else (1 << 64) - s.turn[i]
                # theta^-e and the division are each rounded once in double precision, the table to 2^-64
                assert abs(t / 2.0 ** 64 - rate / (2 * np.pi)) <= 4 * 2.0 ** -53 * rate + 2.0 ** -65
                assert s.axis[i] == a
                i += 1


@pytest.mark.parametrize("kw", [dict(dims=(43, 42, 42)), dict(dims=(64, 64, 2)), dict(dims=(-2, 4, 4)), dict(dims=(4, 4, 4), pairing="half"),
                                dict(dims=(16, 0, 0), theta=0.5), dict(dims=(16, 0, 0), theta=float("nan")),
                                dict(dims=(16, 0, 0), theta=float("inf")), dict(dims=(16, 0, 0), grid=(0, 1)),
                                dict(dims=(16, 0, 0), grid=(1, -3)), dict(dims=(16, 0, 0), pairing="other"), dict(dims=(16, 0))])
def test_plan_refusals(qwm, kw):
    with pytest.raises((qwm.QwmError, ValueError)):
        qwm.RopeSpec(kw.pop("dims"), **kw)


def test_sizes(qwm):
    assert qwm.qwm_window_bytes(8, 2, 3, 4, 5) == (2 * 3 * 9 * 128, 2 * 3 * 9 * 4)
    assert qwm.qwm_window_bytes(4, 2, 3, 0, 5) == (2 * 3 * 5 * 64, 2 * 3 * 5 * 4)
    for bad in ((2, 1, 1, 0, 1), (8, 0, 1, 0, 1), (8, 1, 0, 0, 1), (8, 1, 1, -1, 1), (8, 1, 1, 0, 0),
                (8, 1, 1, 1 << 30, 1 << 30), (8, 256, 256, 0, 1)):
        with pytest.raises(qwm.QwmError):
            qwm.qwm_window_bytes(*bad)


def test_reference_quantiser_bounds():
    """The reference's own properties: |x - s q| <= s / 2, the step is the smallest that covers, and
    packing keeps the values."""
    rng = np.random.default_rng(3)
    for bits in (8, 4):
        x = ref.bf16(rng.standard_normal((64, 128)) * np.exp2(rng.integers(-20, 12, (64, 1))))
        x[0], x[1, :32], x[2] = 0.0, ref.Q[bits] * ref.STEP_TOP[bits], 2.0 ** -30
        x = np.clip(x, -ref.Q[bits] * ref.STEP_TOP[bits], ref.Q[bits] * ref.STEP_TOP[bits])
        q, st = ref.quantise(x, bits)
        s = np.repeat(ref.steps(bits)[st], 32, 1)
        assert np.all(np.abs(x - s * q) <= s / 2)
        lower = np.repeat(ref.steps(bits)[np.maximum(st.astype(int) - 1, 0)], 32, 1)
        worst = np.repeat(np.abs(x).reshape(64, 4, 32).max(-1), 32, 1)
        assert np.all((s == 0) | (lower * ref.Q[bits] < worst))
        assert np.array_equal(ref.values(ref.pack(q, bits), st, bits), s * q)
        v = (s * q).astype(np.float16).astype(np.float64)
        assert np.array_equal(v, s * q)   # exact in fp16


OK = 0x7f00000000   # a stand-in pointer: 16-byte aligned, never read


def _win(qwm, **kw):
    d = dict(bits=8, batch=2, kv_heads=4, reserved=0, sink=4, ring=100, k_codes=OK, v_codes=OK, k_step=OK, v_step=OK)
    d.update(kw)
    return qwm.qwm_window(**d)


def _st(qwm, batch=128 * 8 * 64, head=128, token=128 * 8):
    return qwm.qwm_strides(batch, head, token)


BAD_WINDOWS = [(dict(bits=2), "QWM_ERR_UNSUPPORTED"), (dict(batch=0), "QWM_ERR_ARG"), (dict(kv_heads=-1), "QWM_ERR_ARG"),
               (dict(reserved=1), "QWM_ERR_ARG"), (dict(sink=-1), "QWM_ERR_ARG"), (dict(ring=0), "QWM_ERR_ARG"),
               (dict(ring=1 << 31), "QWM_ERR_SHAPE"), (dict(batch=300, kv_heads=300), "QWM_ERR_SHAPE"),
               (dict(k_codes=None), "QWM_ERR_ARG"), (dict(v_step=None), "QWM_ERR_ARG"), (dict(v_codes=OK + 8), "QWM_ERR_ALIGN"),
               (dict(k_step=OK + 4), "QWM_ERR_ALIGN")]


@pytest.mark.parametrize("kw,err", BAD_WINDOWS)
def test_window_refusals_in_every_call(qwm, kw, err):
    lib, ctx, w, s = qwm.raw_library(), _ctx(qwm), _win(qwm, **kw), _st(qwm)
    want = getattr(qwm, err)
    assert lib.qwm_window_write(ctx, w, OK, s, OK, s, 3, OK, None, None, None, None) == want
    assert lib.qwm_window_read(ctx, w, OK, OK, None, 3, OK, OK, None) == want
    assert lib.qwm_window_attend(ctx, w, OK, s, 3, OK, OK, None, 1, 8, 1.0, OK, s, 0, None, 0, None, 0, None) == want


def test_write_refusals(qwm):
    lib, ctx, w, s = qwm.raw_library(), _ctx(qwm), _win(qwm), _st(qwm)

    def call(ctx=ctx, k=OK, ks=s, v=OK, vs=s, n=3, start=OK, count=None, rope=None, pos=None):
        return lib.qwm_window_write(ctx, w, k, ks, v, vs, n, start, count, rope, pos, None)
    assert call(n=0) == qwm.QWM_OK
    for kw in (dict(ctx=None), dict(n=-1), dict(k=None), dict(v=None), dict(start=None), dict(pos=OK), dict(ks=_st(qwm, head=-8))):
        assert call(**kw) == qwm.QWM_ERR_ARG, kw
    for kw in (dict(k=OK + 2), dict(vs=_st(qwm, token=130)), dict(start=OK + 4), dict(count=OK + 2)):
        assert call(**kw) == qwm.QWM_ERR_ALIGN, kw
    assert call(n=(1 << 24) + 1) == qwm.QWM_ERR_SHAPE
    bad = qwm.RopeSpec((16, 0, 0))
    bad.rot = 130
    assert call(rope=bad) == qwm.QWM_ERR_SHAPE
    bad = qwm.RopeSpec((16, 0, 0))
    bad.axis[3] = 3
    assert call(rope=bad) == qwm.QWM_ERR_ARG


def test_read_refusals(qwm):
    lib, ctx, w = qwm.raw_library(), _ctx(qwm), _win(qwm)
    assert lib.qwm_window_read(ctx, w, OK, OK, None, 0, OK, OK, None) == qwm.QWM_OK
    assert lib.qwm_window_read(ctx, w, OK, OK, None, 3, None, None, None) == qwm.QWM_OK
    assert lib.qwm_window_read(None, w, OK, OK, None, 3, OK, OK, None) == qwm.QWM_ERR_ARG
    assert lib.qwm_window_read(ctx, None, OK, OK, None, 3, OK, OK, None) == qwm.QWM_ERR_ARG
    assert lib.qwm_window_read(ctx, w, None, OK, None, 3, OK, OK, None) == qwm.QWM_ERR_ARG
    assert lib.qwm_window_read(ctx, w, OK, None, None, 3, OK, OK, None) == qwm.QWM_ERR_ARG
    assert lib.qwm_window_read(ctx, w, OK, OK, None, -3, OK, OK, None) == qwm.QWM_ERR_ARG
    assert lib.qwm_window_read(ctx, w, OK, OK, None, 3, OK + 8, OK, None) == qwm.QWM_ERR_ALIGN


def test_attend_refusals(qwm):
    lib, ctx, w, s = qwm.raw_library(), _ctx(qwm), _win(qwm), _st(qwm)

    def call(ctx=ctx, w=w, q=OK, qs=s, nq=3, q_start=OK, length=OK, q_count=None, tpf=1, frames=8, scale=1.0, out=OK, os=s,
             f32=0, lse=None, merge=0, ws=None, nws=0):
        return lib.qwm_window_attend(ctx, w, q, qs, nq, q_start, length, q_count, tpf, frames, scale, out, os, f32, lse,
                                     merge, ws, nws, None)
    assert call(nq=0) == qwm.QWM_OK
    for kw in (dict(ctx=None), dict(nq=-1), dict(q=None), dict(out=None), dict(q_start=None), dict(length=None), dict(tpf=0), dict(frames=0),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(f32=2), dict(merge=2),
               dict(merge=1), dict(merge=1, f32=1), dict(merge=1, lse=OK), dict(os=_st(qwm, token=0)), dict(os=_st(qwm, head=120)),
               dict(os=_st(qwm, batch=128 * 8))):
        assert call(**kw) == qwm.QWM_ERR_ARG, kw
    for kw in (dict(q=OK + 8), dict(out=OK + 4), dict(qs=_st(qwm, head=4)), dict(lse=OK + 2), dict(q_start=OK + 4)):
        assert call(**kw) == qwm.QWM_ERR_ALIGN, kw
    assert call(w=_win(qwm, kv_heads=3)) == qwm.QWM_ERR_SHAPE      # 8 Query heads over 3
    assert call(nq=(1 << 24) + 1) == qwm.QWM_ERR_SHAPE
    assert call(frames=(1 << 31) + 1) == qwm.QWM_ERR_SHAPE
    assert lib.qwm_window_attend_workspace(ctx, _win(qwm, kv_heads=3), 1, 1, 8) == 0


def test_rope_refusals(qwm):
    lib, ctx, s, r = qwm.raw_library(), _ctx(qwm), _st(qwm), qwm.RopeSpec((16, 0, 0))

    def call(ctx=ctx, r=r, x=OK, xs=s, b=2, h=8, n=3, start=OK, pos=None, out=OK + 4096, os=s):
        return lib.qwm_rope(ctx, r, x, xs, b, h, n, start, pos, out, os, None)
    for kw in (dict(n=0), dict(b=0), dict(h=0)):
        assert call(**kw) == qwm.QWM_OK, kw
    for kw in (dict(ctx=None), dict(r=None), dict(x=None), dict(out=None), dict(start=None), dict(n=-1), dict(b=-1),
               dict(out=OK, os=_st(qwm, batch=1 << 20)), dict(os=_st(qwm, token=128)), dict(xs=None)):
        assert call(**kw) == qwm.QWM_ERR_ARG, kw
    for kw in (dict(x=OK + 2), dict(xs=_st(qwm, token=4)), dict(pos=OK + 1)):
        assert call(**kw) == qwm.QWM_ERR_ALIGN, kw
    for kw in (dict(n=(1 << 24) + 1), dict(b=1 << 17), dict(b=60000, n=1 << 20)):
        assert call(**kw) == qwm.QWM_ERR_SHAPE, kw


def test_binding_refuses_host_tensors_and_shapes(qwm):
    import torch

    class Ctx:
        handle, heads, device = None, 8, torch.device("cuda", 0)
    x = torch.zeros(1, 8, 3, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        qwm.qwm_rope(Ctx, qwm.RopeSpec((16, 0, 0)), x, torch.zeros(1, dtype=torch.int64), x)
    with pytest.raises(TypeError):
        qwm.qwm_window_write(Ctx, qwm.Window.empty(8, 1, 8, 0, 4, device="cpu"), x, x, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError):
        qwm.Window.empty(2, 1, 8, 0, 4, device="cpu")


def test_sizes_beyond_the_kernels_index_range_are_refused(qwm):
    for sink, ring in ((0, (1 << 30) + 1), (1 << 29, (1 << 29) + 1), ((1 << 63) - 1, (1 << 63) - 1)):
        with pytest.raises(qwm.QwmError):
            qwm.qwm_window_bytes(8, 1, 1, sink, ring)
    assert qwm.qwm_window_bytes(4, 1, 1, 1 << 29, 1 << 29) == (64 << 30, 4 << 30)
    lib, ctx, w = qwm.raw_library(), _ctx(qwm), _win(qwm)
    for far in (dict(batch=(1 << 38) + 8), dict(head=1 << 62), dict(token=(1 << 63) - 8)):
        assert lib.qwm_window_write(ctx, w, OK, _st(qwm, **far), OK, _st(qwm), 3, OK, None, None, None, None) == qwm.QWM_ERR_ARG
