"""The recent window where its arithmetic is tightest: weights far below a dominating sink, Queries of any
magnitude, infinite channels, far positions; and a layer whose calls are refused or fail half-way."""
import decimal
import math

import numpy as np
import pytest

import window_ref as ref
from test_gpu_window import SCALE, check_attention, ctx_of, f64, fill, ints, rope_bound, rows, spec_args

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qwm():
    import bit_kv_cache_qsac_gb300 as q
    return q


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("sink,other", [(0, 1), (1, -1)])
@pytest.mark.parametrize("gap", [25.0, 23.4])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("nq,heads", [(12, 152), (40, 76), (300, 76)])   # warp tiles; short and full tensor-memory tiles; unsplit
def test_attend_counts_what_a_sink_dominates(qwm, nq, heads, bits, gap, sink, other):
    """One sink above n equal keys by `gap` log2 units, Values `sink` and `other`: a mean weighted by 1 and the
    n keys' share.  Bound: the weights' rounding (2^-11) and grid (2^-32 of the largest, each key), exp2 and
    the logits' scaling (2^-20 and 2^-22 gap), and the fp32 sums, where an addition is off by 2^-24
    (truncated: 2^-23) of the sum, however little is added: the weights are added 64 keys at a time on
    tensor-memory tiles, two at a time in each of 64 lanes on warp tiles, the products 16 keys at a time."""
    n, zero = 1 << 17, {8: 128, 4: 0x88}[bits]
    code = lambda x: zero + x * {8: 1, 4: 0x11}[bits]
    ctx, win = ctx_of(qwm, heads), qwm.Window.empty(bits, 1, heads, 1, n)
    win.k_step.fill_(0x78), win.v_step.fill_(0x78)        # steps of 1
    win.k_codes.fill_(zero), win.v_codes.fill_(code(other))
    win.k_codes[:, :, 0], win.v_codes[:, :, 0] = code(1), code(sink)
    q = torch.ones(1, heads, nq, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(1, heads, nq, 128, dtype=torch.float32, device="cuda")
    lse = torch.empty(1, heads, nq, dtype=torch.float32, device="cuda")
    scale = gap / (128 * math.log2(math.e))
    assert qwm.qwm_window_attend_workspace(ctx, win, nq, 1, n) == 0
    qwm.qwm_window_attend(ctx, win, q, ints([n + 1]), ints([n + 1]), 1, 2 * n, scale, out, lse=lse)
    assert qwm.qwm_sync_status(ctx) == 0
    share = n * 2.0 ** -gap
    want = (sink + share * other) / (1 + share)
    size = (abs(sink) + share * abs(other)) / (1 + share)
    rel = 2.0 ** -11 + 2.0 ** -20 + gap * 2.0 ** -22 + n / 64 * 2.0 ** -24 + n / 16 * 2.0 ** -23
    assert float((out.double() - want).abs().max()) <= size * rel + n * 2.0 ** -32
    assert float((lse.double() - gap - math.log2(1 + share)).abs().max()) <= math.log2(math.e) * n / 64 * 2.0 ** -24 + gap * 2.0 ** -22 + 2.0 ** -20
