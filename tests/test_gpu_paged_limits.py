"""The paged operators where their arithmetic and their loops are tightest: scales and Queries that underflow,
sequences of up to 2^22 tokens."""
import math

import numpy as np
import pytest

import window_ref as ref
from test_gpu_paged import ALL, Batch, attend, ctx_of, f64, gpu_check, ints, rows, starts, status

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qwm():
    import bit_kv_cache_qsac_gb300 as q
    return q


# ------------------------------------------------------------------ attention


@pytest.mark.parametrize("scale", [2.0 ** -20, 1e-10, 1e-30, 1e-45])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("count", [3, 12, 40, 300])   # warp tiles of 8 and 16 rows; short and full tensor-memory tiles
def test_attend_scales_that_underflow(qwm, count, bits, scale):
    """Rows of zeros, rows near the smallest bf16 number and ordinary ones under a mask, at scales that leave all
    logits below 2^-10: every weight is 1 within 2^-9 (e^x for |x| < 2^-10), the mean that of the seen Values, over
    the paged cache and over the window."""
    rng = np.random.default_rng(count + bits)
    n, H = 400, 2
    b = Batch(qwm, rng, bits, 32, H, [n])
    q = rows(rng, H, count, scale=1e-3 if scale > 1e-9 else 1.0, outliers=False)
    q[:, ::3] = 0.0
    q[:, 1::3] = (q[:, 1::3].double() * 2.0 ** -125).to(torch.bfloat16)
    ctx = ctx_of(qwm, H)
    out, lse = torch.zeros(H, count, 128, device="cuda"), torch.zeros(H, count, device="cuda")
    qwm.qwm_paged_attend(ctx, b.pool, b.tab, q, ints([0], torch.int32), ints([count], torch.int32), scale, out, lse=lse, max_count=count)
    win = qwm.Window.empty(bits, 1, H, 0, n)
    for name in ("k_codes", "k_step", "v_codes", "v_step"):   # the same tokens in the window's slots
        pages = getattr(b.pool, name)[b.tab.table[0].long()]
        getattr(win, name)[0] = pages.transpose(0, 1).flatten(1, 2)[:, :n]
    wout, wlse = torch.zeros(1, H, count, 128, device="cuda"), torch.zeros(1, H, count, device="cuda")
    qwm.qwm_window_attend(ctx, win, q[None], ints([n - count]), ints([n]), 1, ALL, scale, wout, lse=wlse)
    assert status(qwm, ctx) == qwm.QWM_OK
    see = torch.arange(n, device="cuda") <= torch.arange(n - count, n, device="cuda")[:, None]
    w = see.double() / see.sum(-1, keepdim=True)
    v = torch.from_numpy(b.v[0]).cuda()
    want, spread, many = w @ v, w @ v.abs(), torch.log2(see.sum(-1).double())
    for o, l in ((out, lse), (wout[0], wlse[0])):
        assert bool(((o.double() - want).abs() <= 2.0 ** -7 * spread).all())
        assert bool(((l.double() - many).abs() <= 2.0 ** -8).all())
