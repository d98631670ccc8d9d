"""Host-side limits of the paged cache (no GPU): the workspace of an attention call."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def qwm():
    import __graft_entry__
    __graft_entry__.build_library()
    import bit_kv_cache_qsac_gb300 as q
    return q


def _ctx(qwm, heads, sms=152):
    """A context's host side: its configuration, a device and its SMs."""
    buf = (C.c_char * 4096)()
    cfg = qwm.qwm_config(heads, 128, 256, 64, 4, 8, 2, 10, 0)
    C.memmove(buf, C.byref(cfg), C.sizeof(cfg))
    C.c_int32.from_buffer(buf, C.sizeof(cfg) + 4).value = sms
    return buf


class _Library:
    """The library with the attention call's own checks of page and workspace in the place of the call."""

    def __init__(self, qwm, real):
        self.qwm, self.real, self.given = qwm, real, []

    def qwm_paged_attend_workspace(self, *a):
        return self.real.qwm_paged_attend_workspace(*a)

    def qwm_paged_attend(self, handle, pool, tab, q, qs, n, first, count, most, *rest):
        need, given = self.real.qwm_paged_attend_workspace(handle, pool, most), rest[-2]
        self.given.append(given)
        if need == 0:
            return self.qwm.QWM_ERR_UNSUPPORTED
        return self.qwm.QWM_ERR_ARG if given < need else self.qwm.QWM_OK


def test_a_refused_call_leaves_later_ones_as_they_are(qwm, monkeypatch):
    """The size that the binding keeps is not that of a refused pool with the same bits, heads and count."""
    import torch

    from bit_kv_cache_qsac_gb300 import paged

    class Ctx:
        handle, heads, device, paged_workspace = _ctx(qwm, 8), 8, torch.device("cpu"), {}
    lib = _Library(qwm, paged._fast)
    monkeypatch.setattr(paged, "_fast", lib)
    monkeypatch.setattr(paged, "_stream_of", lambda ctx, stream: 0)
    q, out = (torch.zeros(8, 3, 128, dtype=torch.bfloat16) for _ in range(2))
    first, count = (torch.tensor([0], dtype=torch.int32) for _ in range(2))

    def call(page):
        pool = qwm.PagePool.empty(8, page, 4, 8, device="cpu")
        qwm.qwm_paged_attend(Ctx, pool, qwm.PageTable.empty(1, 2, page, 4, device="cpu"), q, first, count, 1.0, out)
    with pytest.raises(qwm.QwmError) as e:
        call(24)
    assert e.value.status == qwm.QWM_ERR_UNSUPPORTED
    for _ in range(2):
        call(32)
    assert lib.given[0] == 0 and lib.given[1] == lib.given[2] > 0


@pytest.mark.parametrize("kv", [1, 2, 8])
@pytest.mark.parametrize("group", [1, 3, 8, 16, 32, 33])
def test_workspace_serves_smaller_counts(qwm, kv, group):
    """The bytes for calls of up to max_count new tokens suffice for each smaller count."""
    lib, ctx = qwm.raw_library(), _ctx(qwm, kv * group)
    pool = qwm.qwm_page_pool(8, 64, 40, kv, *[0x7f00000000] * 4)
    sizes = [lib.qwm_paged_attend_workspace(ctx, pool, c) for c in range(1, 80)] + [lib.qwm_paged_attend_workspace(ctx, pool, 1 << 24)]
    assert sizes[0] > 0 and sizes == sorted(sizes)


def test_eps_range(qwm):
    """A mean square of up to 2^113 beside an eps of fp32's largest numbers would be infinite in their sum, and the row 0
    where the formula gives numbers (2^60 / sqrt(2^128) = 2^-4): eps is 2^100 at most."""
    lib, ctx, ok = qwm.raw_library(), _ctx(qwm, 8), 0x7f00000000
    s = qwm.qwm_strides(1 << 14, 128, 1024)
    pool = qwm.qwm_page_pool(8, 64, 40, 8, *[ok] * 4)
    for eps, n, want in ((2.0 ** 100, 0, qwm.QWM_OK), (2.0 ** 100 * (1 + 2.0 ** -23), 0, qwm.QWM_ERR_ARG), (3.4e38, 3, qwm.QWM_ERR_ARG)):
        assert lib.qwm_norm_rope(ctx, None, ok, s, 1, 8, n, None, None, None, None, 0, eps, ok + 4096, s, None) == want
        assert lib.qwm_paged_write(ctx, pool, ok, s, ok, s, n, ok, None, None, None, 1, None, 0, eps, None) == want
