"""The recent window where its arithmetic is tightest: weights far below a dominating sink, Queries of any
magnitude, infinite channels, far positions; and a layer whose calls are refused or fail half-way."""
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


def test_attend_long_caches_in_parts(qwm):
    """A sink above 2^20 equal keys by so much that their weights fall below the fp16 grid: only those of the
    sink's own part (2^18 keys at most) may.  The others' parts carry them in full."""
    n, heads, nq, gap = 1 << 20, 76, 40, 32.5
    ctx, win = ctx_of(qwm, heads), qwm.Window.empty(4, 1, heads, 1, n)
    win.k_step.fill_(0x78), win.v_step.fill_(0x78)        # steps of 1
    win.k_codes.fill_(0x88), win.v_codes.fill_(0x99)
    win.k_codes[:, :, 0], win.v_codes[:, :, 0] = 0x99, 0x88
    q = torch.ones(1, heads, nq, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(1, heads, nq, 128, dtype=torch.float32, device="cuda")
    lse = torch.empty(1, heads, nq, dtype=torch.float32, device="cuda")
    qwm.qwm_window_attend(ctx, win, q, ints([n + 1]), ints([n + 1]), 1, 2 * n, gap / (128 * math.log2(math.e)), out, lse=lse)
    assert qwm.qwm_sync_status(ctx) == 0
    share, part = n * 2.0 ** -gap, 1 << 18
    want = share / (1 + share)
    rel = 2.0 ** -11 + 2.0 ** -20 + gap * 2.0 ** -22 + part / 64 * 2.0 ** -24 + part / 16 * 2.0 ** -23
    assert float((out.double() - want).abs().max()) <= want * rel + part * 2.0 ** -32
    assert float((lse.double() - gap - math.log2(1 + share)).abs().max()) <= math.log2(math.e) * part / 64 * 2.0 ** -24 + gap * 2.0 ** -22 + 2.0 ** -20
    # the parts of a call without a sink: Values 1, -1 and 0 on a half, a quarter and the rest of the keys
    win.k_codes.fill_(0x88), win.v_codes.fill_(0x88)
    win.v_codes[:, :, 1:1 + n // 2], win.v_codes[:, :, 1 + n // 2:1 + 3 * n // 4] = 0x99, 0x77
    qwm.qwm_window_attend(ctx, win, q, ints([n + 1]), ints([n + 1]), 1, 2 * n, 1.0, out, lse=lse)
    want = n / 4 / (n + 1)
    assert float((out.double() - want).abs().max()) <= 0.75 * (part / 64 * 2.0 ** -24 + part / 16 * 2.0 ** -23) + 2.0 ** -20
    assert float((lse.double() - math.log2(n + 1)).abs().max()) <= math.log2(math.e) * part / 64 * 2.0 ** -24 + 2.0 ** -19


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H,kv,nq,length", [(2, 2, 1, 300), (6, 2, 4, 300), (2, 2, 30, 9000), (2, 1, 40, 300), (2, 2, 300, 200), (1, 1, 600, 300)])
def test_attend_queries_of_any_magnitude(qwm, H, kv, nq, length, bits):
    """Rows from 2^-133 to 2^12 beside one another, zero rows and rows with a wide range among them: the
    logits are those of the bf16 Queries within fp32 rounding."""
    rng = np.random.default_rng(nq + bits)
    ctx, win = ctx_of(qwm, H), fill(qwm, ctx_of(qwm, H), rng, bits, kv, 3, length, [length])
    q = rows(rng, 1, H, nq, "token")
    power = torch.tensor([0, -22, -30, 12, -1, -60, 3, -126], device="cuda")[torch.arange(H * nq, device="cuda") % 8]
    q.copy_((q.double() * torch.exp2(power.double()).reshape(1, H, nq, 1)).to(torch.bfloat16))
    if nq > 3:
        q[:, :, 2] = 0
        q[:, :, 3, ::2] *= 2.0 ** -15
    out = torch.empty(1, H, nq, 128, dtype=torch.float32, device="cuda")
    lse = torch.empty(1, H, nq, dtype=torch.float32, device="cuda")
    for scale in (SCALE * 2.0 ** -10, SCALE * 2.0 ** 22):
        use = q if scale < 1 else (q.double() * torch.where(power >= -1, 2.0 ** -24, 1.0).double().reshape(1, H, nq, 1)).to(torch.bfloat16)
        qwm.qwm_window_attend(ctx, win, use, ints([length]), ints([length]), 1, length, scale, out, lse=lse)
        assert qwm.qwm_sync_status(ctx) == 0
        check_attention(win, use, [length], [length], 1, length, scale, out, lse, out_eps=2.0 ** -22)


# ------------------------------------------------------------------ rotary positions

@pytest.mark.parametrize("start", [2 ** 33, 2 ** 40 + 12345, 2 ** 47 - 1])
@pytest.mark.parametrize("pairing", ["interleaved", "half"])
def test_rope_far_positions(qwm, pairing, start):
    """Against angles of 200 bits: beside the rounding, a position's angle is off by at most 2^-65 turns a
    position (the table's rounding)."""
    kw = dict(dims=(128, 0, 0), theta=500000.0, pairing=pairing)
    rng = np.random.default_rng(start % 1000)
    h, n = 3, 40
    x = rows(rng, 1, h, n)
    out = torch.empty(1, h, n, 128, dtype=torch.bfloat16, device="cuda")
    qwm.qwm_rope(ctx_of(qwm, h), qwm.RopeSpec(**kw), x, ints([start]), out)
    dims, theta, _, shared = spec_args(kw)
    turns = ref.exact_turns(dims, theta, shared)
    part = np.array([[((start + i) * t % 2 ** 200 >> 140) / 2.0 ** 60 for t in turns] for i in range(n)])
    c, s = np.cos(2 * np.pi * part), np.sin(2 * np.pi * part)
    at = (np.arange(64) * 2, np.arange(64) * 2 + 1) if pairing == "interleaved" else (np.arange(64), np.arange(64) + 64)
    for j in range(h):
        src, want, pair = f64(x[0, j]), np.zeros((n, 128)), np.zeros((n, 128))
        p, q = src[:, at[0]], src[:, at[1]]
        want[:, at[0]], want[:, at[1]] = p * c - q * s, p * s + q * c
        pair[:, at[0]] = pair[:, at[1]] = np.abs(p) + np.abs(q)
        far = (start + n) * 2.0 ** -65 * 2 * np.pi
        assert np.all(np.abs(f64(out[0, j]) - want) <= rope_bound(src, want, kw) + far * pair)


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
def test_rope_cosine_and_sine(qwm, pairing):
    """Rows (a, b) that nearly cancel, a cos = b sin to a few parts in 2^16, show the angles' cosine and sine to
    2^-28: the result's own roundings (2^-8 to bf16, 2^-23 before) are relative to what is left."""
    spec = qwm.RopeSpec((128, 0, 0), theta=1000.0, pairing=pairing)
    n, turn = 4096, np.array(spec.turn[:], np.uint64)
    start = 77_777
    whole = (np.arange(start, start + n, dtype=np.uint64)[:, None] * turn)   # modulo 2^64
    ang = whole.astype(np.longdouble) * (2 * np.arctan2(np.longdouble(0), np.longdouble(-1)) / np.longdouble(2) ** 64)
    c, s = np.cos(ang), np.sin(ang)
    small, large = np.abs(s).astype(np.float64), np.abs(c).astype(np.float64)
    left, best = np.full((n, 64), np.inf), np.zeros((2, n, 64))
    for m in range(128, 256):   # a of 8 bits, b the nearest of 8 bits to a cos / sin
        b = ref.bf16(m * large / np.maximum(small, 1e-9))
        d = np.abs(m * large - b * small) / (m + b)
        pick = d < left
        left[pick], best[0][pick], best[1][pick] = d[pick], m, b[pick]
    a, b = best[0] * np.sign(c).astype(np.float64), best[1] * np.sign(s).astype(np.float64)   # a c - b s cancels
    at = (np.arange(64) * 2, np.arange(64) * 2 + 1) if pairing == "interleaved" else (np.arange(64), np.arange(64) + 64)
    x = np.zeros((n, 128))
    x[:, at[0]], x[:, at[1]] = a, b
    t = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()[None, None]
    out = torch.empty_like(t)
    qwm.qwm_rope(ctx_of(qwm, 1), spec, t, ints([start]), out)
    want = (a * c - b * s).astype(np.float64)
    got = f64(out[0, 0])[:, at[0]]
    pair = np.abs(a) + np.abs(b)
    assert np.median(np.abs(want) / pair) < 2.0 ** -14   # they do cancel
    assert np.all(np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + 2.0 ** -28 * pair)
    # the other channel of each pair: a s + b c, with b and a exchanged in sign
    y = np.zeros((n, 128))
    y[:, at[0]], y[:, at[1]] = -b, a
    t = torch.from_numpy(y.astype(np.float32)).to(torch.bfloat16).cuda()[None, None]
    qwm.qwm_rope(ctx_of(qwm, 1), spec, t, ints([start]), out)
    assert np.all(np.abs(f64(out[0, 0])[:, at[1]] - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + 2.0 ** -28 * pair)


BAD = [(np.inf, 1.0), (1.0, np.inf), (-np.inf, 0.5), (np.inf, np.inf), (np.inf, -np.inf), (-np.inf, -np.inf), (np.nan, 1.0), (2.0, np.nan),
       (np.inf, np.nan), (3.0e38, 3.0e38), (3.0e38, -3.0e38)]


def with_bad_pairs(rng, pairing, R, n):
    """Rows of noise; row i has the pair BAD[i % len(BAD)] at pair i % (R / 2)."""
    x = ref.bf16(rng.standard_normal((n, 128)))
    at = []
    for i in range(n):
        j = (7 * i) % (R // 2)
        at.append((2 * j, 2 * j + 1) if pairing == "interleaved" else (j, j + R // 2))
        x[i, at[i][0]], x[i, at[i][1]] = BAD[i % len(BAD)]
    return x, at


def same_class(got, want):
    return (np.isnan(got) and np.isnan(want)) or (np.isinf(want) and got == want) or (np.isfinite(want) and np.isfinite(got))


@pytest.mark.parametrize("pairing,dims", [("interleaved", (44, 42, 42)), ("interleaved", (2, 4, 30)), ("half", (128, 0, 0)), ("half", (16, 0, 16))])
@pytest.mark.parametrize("start", [0, 1234])
def test_rope_infinite_channels(qwm, pairing, dims, start):
    """An infinite or NaN channel gives its pair what the formula gives (an angle of 0 has a sine of 0, and 0
    times infinity is NaN), sums beyond the range are infinite, and no other channel is touched."""
    kw = dict(dims=dims, theta=100.0, pairing=pairing)
    rng = np.random.default_rng(3)
    n = 33
    x, at = with_bad_pairs(rng, pairing, sum(dims), n)
    t = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()[None, None]
    clean = t.clone()
    for i in range(n):
        clean[0, 0, i, list(at[i])] = 1.0
    out, base = torch.empty_like(t), torch.empty_like(t)
    qwm.qwm_rope(ctx_of(qwm, 1), qwm.RopeSpec(**kw), t, ints([start]), out)
    qwm.qwm_rope(ctx_of(qwm, 1), qwm.RopeSpec(**kw), clean, ints([start]), base)
    src = f64(t[0, 0])
    with np.errstate(invalid="ignore", over="ignore"):
        want = ref.rope(src, *spec_args(kw), ref.grid_positions(start, n, 1, 1))
    want = np.where(np.abs(want) >= 2.0 ** 128 * (1 - 2.0 ** -9), np.sign(want) * np.inf, want)
    got = f64(out[0, 0])
    for i in range(n):
        for ch in at[i]:
            assert same_class(got[i, ch], want[i, ch]), (i, ch, src[i, list(at[i])], got[i, ch], want[i, ch])
        out[0, 0, i, list(at[i])] = base[0, 0, i, list(at[i])]
    assert torch.equal(out, base)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("pairing", ["interleaved", "half"])
def test_write_cuts_infinite_channels_after_turning(qwm, bits, pairing):
    kw = dict(dims=(128, 0, 0), theta=100.0, pairing=pairing)
    top = ref.Q[bits] * ref.STEP_TOP[bits]
    rng = np.random.default_rng(4)
    n = 2 * len(BAD)
    x, at = with_bad_pairs(rng, pairing, 128, n)
    t = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()[None, None]
    ctx, win = ctx_of(qwm, 1), qwm.Window.empty(bits, 1, 1, 0, n)
    qwm.qwm_window_write(ctx, win, t, torch.zeros_like(t), ints([50]), rope=qwm.RopeSpec(**kw))
    assert qwm.qwm_sync_status(ctx) == qwm.QWM_ERR_RANGE
    kh, vh = torch.empty_like(t), torch.empty_like(t)
    qwm.qwm_window_read(ctx, win, ints([50]), ints([50 + n]), kh, vh)
    with np.errstate(invalid="ignore", over="ignore"):
        want = ref.rope(f64(t[0, 0]), *spec_args(kw), ref.grid_positions(50, n, 1, 1))
    want = np.where(np.isnan(want), 0.0, np.clip(want, -top, top))
    got = f64(kh[0, 0])
    for i in range(n):
        for ch in at[i]:
            assert got[i, ch] == want[i, ch] or abs(got[i, ch] - want[i, ch]) <= 2.0 ** -8 * abs(want[i, ch]), (i, ch, got[i, ch], want[i, ch])


# ------------------------------------------------------------------ the layer

def tiny_stream(n, steps, heads=2):
    import synth
    from helpers import from_u16
    keys, vals = synth.keys(synth.TINY), synth.values(synth.TINY)
    cut = lambda x, t: from_u16(np.ascontiguousarray(x[:, (t * n) % 1024:(t * n) % 1024 + n]), torch.bfloat16)
    return [(cut(keys, t), cut(vals, t), from_u16(synth.queries(synth.TINY, t, n), torch.bfloat16)) for t in range(steps)]


def state_of(layer):
    """What a layer holds, without the slots of the chunk that was not added."""
    return [layer.length, len(layer.packed.chunks), layer.packed.n_seen, layer.packed.S.clone(), layer.packed.n.clone(), layer.packed.w.clone()]


def same_state(a, b):
    return all(torch.equal(x, y) if isinstance(x, torch.Tensor) else x == y for x, y in zip(a, b))


@pytest.mark.parametrize("rope", [False, True])
def test_layer_takes_queries_of_any_strides(qwm, rope):
    from bit_kv_cache_qsac_gb300 import stream
    n, ctx = 256, qwm.Context(heads=2, n_centroids=64)
    spec = qwm.RopeSpec((44, 42, 42), grid=(16, 16)) if rope else None
    a, b = (stream.WindowedLayer(ctx, n, 2, tpf=64, rope=spec) for _ in range(2))
    for k, v, q in tiny_stream(n, 4):
        major = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)   # as a projection leaves it
        assert torch.equal(a.step(k, v, q), b.step(major(k), major(v), major(q)))
    assert same_state(state_of(a), state_of(b)) and a.check() == 0


def refused(k, v, q):
    """Steps that must be refused, one wrong operand each."""
    half = lambda t: t.to(torch.float16)
    every_other = lambda t: torch.zeros(*t.shape[:2], 256, dtype=t.dtype, device=t.device)[..., ::2]
    odd = lambda t: torch.zeros(t.shape[0], t.shape[1], 132, dtype=t.dtype, device=t.device)[..., :128]
    off = lambda t: torch.zeros(t.numel() + 8, dtype=t.dtype, device=t.device)[4:4 + t.numel()].view(t.shape)
    for bad in (half, every_other, odd, off, lambda t: t.cpu(), lambda t: t[:1], lambda t: t[..., :64], lambda t: t[0], lambda t: None):
        yield bad(k), v, q
        yield k, bad(v), q
        yield k, v, bad(q)
    yield k[:, :-1], v, q
    yield k, v[:, :-1], q
    yield k, v, torch.cat([q, q], 1)


@pytest.mark.parametrize("rope", [False, True])
def test_layer_refused_steps_change_nothing(qwm, rope):
    from bit_kv_cache_qsac_gb300 import stream
    n, ctx = 256, qwm.Context(heads=2, n_centroids=64)
    spec = qwm.RopeSpec((44, 42, 42), grid=(16, 16)) if rope else None
    a, b = (stream.WindowedLayer(ctx, n, 2, tpf=64, rope=spec) for _ in range(2))
    for k, v, q in tiny_stream(n, 4):   # with room in the window, with a full one, over a packed history
        before = state_of(b) + [b.window.k_codes.clone(), b.window.v_codes.clone()]
        for args in refused(k, v, q):
            with pytest.raises((TypeError, ValueError)):
                b.step(*args)
        assert same_state(before, state_of(b) + [b.window.k_codes, b.window.v_codes])
        assert torch.equal(a.step(k, v, q), b.step(k, v, q))
    assert same_state(state_of(a), state_of(b))


@pytest.mark.parametrize("call", ["qwm_window_read", "qwm_fit_centroids_kv", "qwm_quantize_kv", "qwm_window_write", "qwm_rope",
                                  "qwm_attend_merge", "qwm_window_attend", "qwm_update_query_stats"])
def test_layer_repeats_a_step_that_failed_half_way(qwm, call, monkeypatch):
    """Whichever call of a step reports an error, the step may be made again, and the layer goes on as if
    it had succeeded at once."""
    from bit_kv_cache_qsac_gb300 import stream
    n, ctx = 256, qwm.Context(heads=2, n_centroids=64)
    spec = qwm.RopeSpec((44, 42, 42), grid=(16, 16))
    a, b = (stream.WindowedLayer(ctx, n, 2, tpf=64, rope=spec) for _ in range(2))
    real, failed = getattr(stream, call), 0
    for k, v, q in tiny_stream(n, 5):
        want = a.step(k, v, q)

        def fails(*args, **kw):
            raise qwm.QwmError(qwm.QWM_ERR_CUDA, call)
        monkeypatch.setattr(stream, call, fails)
        length = b.length
        try:
            got = b.step(k, v, q)
        except qwm.QwmError:
            failed += 1
            assert b.length == length
            monkeypatch.setattr(stream, call, real)
            got = b.step(k, v, q)
        monkeypatch.setattr(stream, call, real)
        assert torch.equal(got, want)
        assert same_state(state_of(a), state_of(b))
    assert failed >= 3


def test_layer_over_more_chunks_than_one_call_takes(qwm):
    """qwm_attend_merge takes 128 chunks; the layer's history may be longer."""
    from bit_kv_cache_qsac_gb300 import stream
    n, H, ctx = 64, 2, qwm.Context(heads=2, n_centroids=64, kmeans_iters=1)
    layer = stream.WindowedLayer(ctx, n, 1)
    data = tiny_stream(n, 132)
    for k, v, q in data:
        out = layer.step(k, v, q)
    assert len(layer.packed.chunks) == 131 and layer.check() == 0
    # the same by hand: every chunk's part, joined by the log-sum-exps in 64 bits
    parts = []
    for c in layer.packed.chunks:
        o, s = torch.empty(H, n, 128, device="cuda"), torch.empty(H, n, device="cuda")
        qwm.qwm_attend_merge(ctx, q, n, [c], SCALE, o, s, False)
        parts.append((o.double(), s.double()))
    o, s = torch.empty(1, H, n, 128, device="cuda"), torch.empty(1, H, n, device="cuda")
    qwm.qwm_window_attend(ctx, layer.window, q[None], ints([131 * n]), ints([132 * n]), n, 3, SCALE, o, lse=s)
    parts.append((o[0].double(), s[0].double()))
    top = torch.stack([s for _, s in parts]).amax(0)
    w = [torch.exp2(s - top)[..., None] for _, s in parts]
    want = sum(x * y for x, (y, _) in zip(w, parts)) / sum(w)
    # the weights' fp16 rounding in every part (2^-11 each, on numerator and denominator), against |V| within
    # the attention's bar
    assert float((out.double() - want).abs().max() / want.pow(2).mean().sqrt()) <= 2e-2


@pytest.mark.parametrize("fails", [False, True])
def test_layer_on_other_streams_than_its_own(qwm, fails, monkeypatch):
    """Built behind work on one stream, stepped on others in turn (after a step that failed on the one, on
    the other): every step waits for what it needs."""
    from bit_kv_cache_qsac_gb300 import stream
    n, ctx = 256, qwm.Context(heads=2, n_centroids=64)
    data = tiny_stream(n, 6)
    plain = stream.WindowedLayer(ctx, n, 2, tpf=64)
    want = [plain.step(*d) for d in data]
    busy, others = torch.cuda.Stream(), [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    with torch.cuda.stream(busy):
        torch.cuda._sleep(20_000_000)   # about 10 ms before the layer's tensors are filled
        layer = stream.WindowedLayer(ctx, n, 2, tpf=64)

    def broken(*args, **kw):
        raise qwm.QwmError(qwm.QWM_ERR_CUDA, "qwm_window_attend")
    got = []
    for i, d in enumerate(data):
        for s in others:
            with torch.cuda.stream(s):
                torch.cuda._sleep(2_000_000 * (1 + i % 2))
        if fails:
            with monkeypatch.context() as m, pytest.raises(qwm.QwmError):
                m.setattr(stream, "qwm_window_attend", broken)
                layer.step(*d, stream=others[i % 2])
        got.append(layer.step(*d, stream=others[(i + fails) % 2]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_layer_step_captured_in_a_graph(qwm):
    """A step with room in the window captured on a stream of its own and replayed with other operands."""
    from bit_kv_cache_qsac_gb300 import stream
    n, ctx = 256, qwm.Context(heads=2, n_centroids=64)
    (k0, v0, q0), (k1, v1, q1) = tiny_stream(n, 2)
    plain, layer = (stream.WindowedLayer(ctx, n, 2, tpf=64) for _ in range(2))
    plain.step(k0, v0, q0), layer.step(k0, v0, q0)
    want = plain.step(k1, v1, q1)
    k, v, q = k0.clone(), v0.clone(), q0.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(k, v, q)
    k.copy_(k1), v.copy_(v1), q.copy_(q1)
    graph.replay()
    assert torch.equal(out, want) and torch.equal(layer.window.k_codes, plain.window.k_codes)
    torch.cuda.synchronize()
    assert layer.length == 2 * n and torch.equal(layer.packed.S, plain.packed.S)
