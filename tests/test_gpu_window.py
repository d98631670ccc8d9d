"""The recent window on the GPU against the 64-bit reference: rotary positions, the window cache
(written and read back), attention over it, and runs of them together."""
import math

import numpy as np
import pytest

import window_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)


@pytest.fixture(scope="module")
def qwm():
    import bit_kv_cache_qsac_gb300 as q
    return q


_CTX = {}


def ctx_of(qwm, heads):
    if heads not in _CTX:
        _CTX[heads] = qwm.Context(heads=heads)
    return _CTX[heads]


def rows(rng, b, h, n, layout="token", scale=1.0, outliers=True):
    """bf16 activations [b][h][n][128], token-major or head-major memory."""
    x = rng.standard_normal((b, h, n, 128)).astype(np.float32) * scale
    if outliers:
        x[..., rng.permutation(128)[:8]] *= 4
    t = torch.from_numpy(x).to(torch.bfloat16).cuda()
    if layout == "token":
        t = t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    elif layout == "padded":   # rows 160 elements apart
        big = torch.full((b, h, n, 160), 9.0, dtype=torch.bfloat16, device="cuda")
        big[..., :128] = t
        t = big[..., :128]
    return t


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def ints(v, dtype=torch.int64):
    return torch.tensor(v, dtype=dtype, device="cuda")


# ------------------------------------------------------------------ rotary positions

SPECS = {"video": dict(dims=(44, 42, 42), theta=10000.0, pairing="interleaved", grid=(45, 80)),
         "text": dict(dims=(128, 0, 0), theta=1e6, pairing="half"),
         "shared": dict(dims=(32, 48, 48), theta=(1e4, 1e3, 50.0), pairing="half", shared_freq=True, grid=(7, 3)),
         "partial": dict(dims=(16, 0, 16), theta=256.0, pairing="half", grid=(2, 9)),
         "odd": dict(dims=(2, 4, 30), theta=100.0, pairing="interleaved", grid=(5, 5)),
         "none": dict(dims=(0, 0, 0), pairing="interleaved")}


def spec_args(kw):
    th = kw.get("theta", 10000.0)
    return kw["dims"], th if isinstance(th, tuple) else (th,) * 3, kw["pairing"], kw.get("shared_freq", False)


def rope_bound(x, want, kw):
    """A result is a c - b s in fp32 with the products' errors carried (cos and sin within 2^-26 of the
    true ones, the sum rounded once: under 2^-24 of |a| + |b|), then rounded to bf16 (2^-8 relative)."""
    pair = np.zeros_like(x)
    R, half = sum(kw["dims"]), sum(kw["dims"]) // 2
    for i in range(half):
        c = (2 * i, 2 * i + 1) if kw["pairing"] == "interleaved" else (i, i + half)
        pair[..., c[0]] = pair[..., c[1]] = np.abs(x[..., c[0]]) + np.abs(x[..., c[1]])
    return 2.0 ** -8 * np.abs(want) + 2.0 ** -23 * pair


@pytest.mark.parametrize("name", SPECS)
@pytest.mark.parametrize("b,h,n,layout,start", [(1, 3, 1, "token", 0), (2, 5, 37, "head", 1000), (3, 1, 16, "padded", 3_000_000_000),
                                                (1, 40, 65, "token", 75_600)])
def test_rope(qwm, name, b, h, n, layout, start):
    kw = SPECS[name]
    rng = np.random.default_rng(b * 100 + n)
    x = rows(rng, b, h, n, layout)
    starts = [start + 11 * i for i in range(b)]
    out = torch.empty(b, h, n, 128, dtype=torch.bfloat16, device="cuda")
    qwm.qwm_rope(ctx_of(qwm, h), qwm.RopeSpec(**kw), x, ints(starts), out)
    dims, theta, pairing, shared = spec_args(kw)
    xr, got = f64(x), f64(out)
    for i in range(b):
        pos = ref.grid_positions(starts[i], n, *kw.get("grid", (1, 1)))
        for j in range(h):
            want = ref.rope(xr[i, j], dims, theta, pairing, shared, pos)
            assert np.all(np.abs(got[i, j] - want) <= rope_bound(xr[i, j], want, kw))
    keep = sum(dims)
    assert torch.equal(out[..., keep:], x[..., keep:])


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
def test_rope_explicit_positions_in_place_and_skipped_sequences(qwm, pairing):
    kw = dict(dims=(48, 32, 32), theta=500.0, pairing=pairing)
    rng = np.random.default_rng(7)
    x = rows(rng, 3, 4, 21, "token")
    keep = x.clone()
    pos = ints(rng.integers(-(2 ** 31), 2 ** 31, (3, 21, 3)).tolist(), torch.int32)
    qwm.qwm_rope(ctx_of(qwm, 4), qwm.RopeSpec(**kw), x, ints([0, -1, 5]), x, pos=pos)
    dims, theta, _, shared = spec_args(kw)
    assert torch.equal(x[1], keep[1])
    for i in (0, 2):
        for j in range(4):
            src = f64(keep[i, j])
            want = ref.rope(src, dims, theta, pairing, shared, pos[i].cpu().numpy().astype(np.int64))
            assert np.all(np.abs(f64(x[i, j]) - want) <= rope_bound(src, want, kw))


@pytest.mark.parametrize("name", ["video", "shared", "partial"])
def test_rope_inverse_is_the_gradient(qwm, name):
    """d<w, rope(x)>/dx = inverse rope(w): against the formula, and against differences of the 64-bit
    rotation."""
    kw = SPECS[name]
    rng = np.random.default_rng(9)
    w = rows(rng, 1, 2, 9, "head")
    g = torch.empty_like(w)
    qwm.qwm_rope(ctx_of(qwm, 2), qwm.RopeSpec(**kw, inverse=True), w, ints([123]), g)
    dims, theta, pairing, shared = spec_args(kw)
    pos = ref.grid_positions(123, 9, *kw.get("grid", (1, 1)))
    for j in range(2):
        wj = f64(w[0, j])
        want = ref.rope(wj, dims, theta, pairing, shared, pos, sign=-1.0)
        bound = rope_bound(wj, want, kw)
        assert np.all(np.abs(f64(g[0, j]) - want) <= bound)
        x = rng.standard_normal((9, 128))
        for c in (0, 1, 17, 63, 127):
            d = np.zeros((9, 128))
            d[:, c] = 0.5   # the rotation is linear: the difference is exact up to 64-bit rounding
            diff = (wj * (ref.rope(x + d, dims, theta, pairing, shared, pos) - ref.rope(x - d, dims, theta, pairing, shared, pos))).sum(1)
            assert np.all(np.abs(f64(g[0, j])[:, c] - diff) <= bound[:, c] + 1e-12)


# ------------------------------------------------------------------ the window cache

def check_written(win, b, h, slot, want_q, want_step, key):
    codes = (win.k_codes if key else win.v_codes)[b, h, slot].cpu().numpy()
    step = (win.k_step if key else win.v_step)[b, h, slot].cpu().numpy()
    assert np.array_equal(step, want_step)
    assert np.array_equal(codes, ref.pack(want_q, win.bits))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("b,h,n,sink,ring,starts,counts", [
    (1, 1, 1, 0, 1, [0], None), (1, 2, 1, 4, 9, [30], None), (2, 3, 50, 5, 64, [0, 3], None),
    (3, 2, 70, 3, 33, [1, 40, 1000], [70, 0, 55]),       # more tokens than slots: the last ones stay
    (2, 1, 16, 40, 7, [-1, 30], [16, 16]), (1, 4, 129, 0, 300, [5_000_000_000], None)])
def test_write_codes_exactly(qwm, bits, b, h, n, sink, ring, starts, counts):
    rng = np.random.default_rng(n + bits)
    k, v = rows(rng, b, h, n, "token"), rows(rng, b, h, n, "padded", scale=0.02)
    ctx, win = ctx_of(qwm, h), qwm.Window.empty(bits, b, h, sink, ring)
    for t in (win.k_codes, win.v_codes, win.k_step, win.v_step):
        t.fill_(0xAB)
    qwm.qwm_window_write(ctx, win, k, v, ints(starts), count=ints(counts, torch.int32) if counts else None)
    assert qwm.qwm_sync_status(ctx) == 0
    touched = np.zeros((b, sink + ring), bool)
    for i in range(b):
        m = counts[i] if counts else n
        if starts[i] < 0:
            m = 0
        last = {}
        for j in range(m):
            last[ref.slot_of(starts[i] + j, sink, ring)] = j
        slots, src = list(last), list(last.values())
        touched[i, slots] = True
        if not slots:
            continue
        for hh in range(h):
            for x, key in ((k, True), (v, False)):
                q, st = ref.quantise(f64(x[i, hh])[src], bits)
                check_written(win, i, hh, slots, q, st, key)
    left = torch.from_numpy(~touched).cuda()
    for t in (win.k_codes, win.v_codes, win.k_step, win.v_step):
        assert bool((t.transpose(1, 2)[left] == 0xAB).all())   # every other slot as it was


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("name", ["video", "text", "partial"])
def test_write_turns_keys_as_rope_does(qwm, bits, name):
    rng = np.random.default_rng(21)
    spec = qwm.RopeSpec(**SPECS[name])
    k, v = rows(rng, 2, 5, 83), rows(rng, 2, 5, 83)
    start, ctx = ints([17, 40_000]), ctx_of(qwm, 5)
    a, c = qwm.Window.empty(bits, 2, 5, 2, 90), qwm.Window.empty(bits, 2, 5, 2, 90)
    qwm.qwm_window_write(ctx, a, k, v, start, rope=spec)
    turned = torch.empty(2, 5, 83, 128, dtype=torch.bfloat16, device="cuda")
    qwm.qwm_rope(ctx, spec, k, start, turned)
    qwm.qwm_window_write(ctx, c, turned, v, start)
    for x, y in ((a.k_codes, c.k_codes), (a.k_step, c.k_step), (a.v_codes, c.v_codes), (a.v_step, c.v_step)):
        assert torch.equal(x, y)
    pos = ints(rng.integers(0, 50, (2, 83, 3)).tolist(), torch.int32)
    qwm.qwm_window_write(ctx, a, k, v, start, rope=spec, pos=pos)
    qwm.qwm_rope(ctx, spec, k, start, turned, pos=pos)
    qwm.qwm_window_write(ctx, c, turned, v, start)
    assert torch.equal(a.k_codes, c.k_codes) and torch.equal(a.k_step, c.k_step)


@pytest.mark.parametrize("bits", [8, 4])
def test_write_extremes(qwm, bits):
    """Zero rows, tiny and largest values, ties; out of range, infinite and NaN elements are cut and
    recorded, and touch no other group."""
    top = ref.Q[bits] * ref.STEP_TOP[bits]
    rng = np.random.default_rng(4)
    x = ref.bf16(rng.standard_normal((12, 128)))
    x[0] = 0.0
    x[1] = ref.bf16(x[1] * 2.0 ** -30)
    x[2, :32] = ref.bf16(np.linspace(-top, top, 32))
    x[2] = np.clip(x[2], -top, top)
    x[3] = ref.Q[bits]
    x[3, ::2] = np.arange(64) % ref.Q[bits] + 0.5     # exact halves at step 1
    x[4] = 2.0 ** -126
    x[5] = -x[3]
    good = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()[None, None]
    ctx, win = ctx_of(qwm, 1), qwm.Window.empty(bits, 1, 1, 0, 12)
    qwm.qwm_window_write(ctx, win, good, good, ints([0]))
    assert qwm.qwm_sync_status(ctx) == 0
    q, st = ref.quantise(f64(good[0, 0]), bits)
    check_written(win, 0, 0, list(range(12)), q, st, True)
    bad = good.clone()
    bad[0, 0, 6, 3], bad[0, 0, 7, 40], bad[0, 0, 8, 127], bad[0, 0, 9, 64] = float("nan"), float("inf"), -float("inf"), 3e38
    qwm.qwm_window_write(ctx, win, good, bad, ints([0]))
    assert qwm.qwm_sync_status(ctx) == qwm.QWM_ERR_RANGE and qwm.qwm_sync_status(ctx) == 0
    cut = np.clip(np.nan_to_num(f64(bad[0, 0]), nan=0.0, posinf=1e30, neginf=-1e30), -top, top)
    q, st = ref.quantise(cut, bits)
    check_written(win, 0, 0, list(range(12)), q, st, False)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("sink,ring,length,start,n,counts", [(0, 1, 1, 0, 1, None), (3, 20, 100, 60, 50, None), (5, 40, 30, 0, 33, [20]),
                                                             (0, 64, 64, -2, 5, None), (130, 7, 50, 10, 200, [199])])
def test_read_back(qwm, bits, sink, ring, length, start, n, counts):
    rng = np.random.default_rng(ring)
    ctx, win = ctx_of(qwm, 2), qwm.Window.empty(bits, 1, 2, sink, ring)
    k, v = rows(rng, 1, 2, length), rows(rng, 1, 2, length)
    qwm.qwm_window_write(ctx, win, k, v, ints([0]))
    kh, vh = (torch.full((1, 2, n, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cnt = ints(counts, torch.int32) if counts else None
    qwm.qwm_window_read(ctx, win, ints([start]), ints([length]), kh, vh, count=cnt)
    m = 0 if start < 0 else (counts[0] if counts else n)
    have = set(ref.held(length, sink, ring))
    for x, got in ((k, kh), (v, vh)):
        for h in range(2):
            q, st = ref.quantise(f64(x[0, h]), bits)
            val = ref.values(ref.pack(q, bits), st, bits)
            g = f64(got[0, h])
            for i in range(n):
                p = start + i
                want = np.full(128, 7.0) if i >= m else (ref.bf16(val[p]) if p in have else np.zeros(128))
                assert np.array_equal(g[i], want), (i, p)
    only = torch.zeros_like(kh)
    qwm.qwm_window_read(ctx, win, ints([max(start, 0)]), ints([length]), None, only)
    if start >= 0:
        assert torch.equal(only[:, :, :m], vh[:, :, :m])


# ------------------------------------------------------------------ attention

def fill(qwm, ctx, rng, bits, kv, sink, ring, lengths, scale_k=1.0):
    """A window written token block by token block up to lengths[b], and its decoded rows by position."""
    b = len(lengths)
    win = qwm.Window.empty(bits, b, kv, sink, ring)
    n = max(max(lengths), 1)
    k, v = rows(rng, b, kv, n, scale=scale_k), rows(rng, b, kv, n)
    done = 0
    while done < n:
        m = min(max(1, n // 3), n - done)
        cnt = [min(m, max(0, L - done)) for L in lengths]
        qwm.qwm_window_write(ctx, win, k[:, :, done:done + m], v[:, :, done:done + m], ints([done] * b), count=ints(cnt, torch.int32))
        done += m
    return win


def decoded(win, i, h, length):
    pos = np.array(ref.held(length, win.sink, win.ring), np.int64)
    slots = [ref.slot_of(int(p), win.sink, win.ring) for p in pos]
    out = []
    for c, s in ((win.k_codes, win.k_step), (win.v_codes, win.v_step)):
        out.append(ref.values(c[i, h].cpu().numpy()[slots], s[i, h].cpu().numpy()[slots], win.bits))
    return pos, out[0], out[1]


def check_attention(win, q, q_starts, lengths, tpf, frames, scale, out, lse, counts=None, out_eps=2.0 ** -8):
    """Against the reference, within: the logits' fp32 sums (128 products and a scaling: 2^-16 of their
    magnitude A in log2 units, so weights are off by that too), the weights' rounding to fp16 (2^-11,
    and 2^-25 absolute below its normal range, against a largest weight of at least 1), exp2 (2^-20),
    each on numerator and denominator; the output's own rounding."""
    b, H, nq, _ = q.shape
    g = H // win.kv_heads
    for i in range(b):
        live = 0 if q_starts[i] < 0 else (counts[i] if counts else nq)
        if live == 0:
            continue
        for h in range(H):
            pos, k, v = decoded(win, i, h // g, lengths[i])
            want, wl, mag, spread = ref.attend(f64(q[i, h])[:live], k, v, pos, q_starts[i], tpf, frames, win.sink, scale)
            got, gl = f64(out[i, h])[:live], lse[i, h].double().cpu().numpy()[:live]
            none = np.isneginf(wl)
            assert np.array_equal(none, np.isneginf(gl)), (i, h)
            assert np.all(got[none] == 0)
            eps = (2.0 ** -11 + 2.0 ** -16 * mag + 2.0 ** -20)[:, None]
            bound = 2 * eps * spread + len(pos) * 2.0 ** -25 * (np.abs(v).max() if len(v) else 0) + out_eps * np.abs(want)
            assert np.all(np.abs(got - want) <= bound), (i, h, np.max(np.abs(got - want) / bound))
            d = np.abs(gl[~none] - wl[~none])
            assert np.all(d <= 2.0 ** -16 * mag[~none] + 2.0 ** -20 + 2.0 ** -22 * np.abs(wl[~none])), (i, h, d.max())


# (bits, lengths, H, kv, nq, sink, ring, tpf, frames)
FEW = [(8, [1], 1, 1, 1, 0, 1, 1, 1), (4, [1], 1, 1, 1, 1, 1, 1, 5), (8, [200], 8, 2, 1, 4, 100, 1, 100),
       (4, [300, 0, 17, 150], 6, 2, 5, 3, 150, 1, 120), (8, [40, 41], 4, 4, 7, 8, 33, 1, 10),
       (4, [500], 16, 1, 1, 0, 500, 1, 500), (8, [500], 15, 1, 1, 7, 400, 1, 77), (4, [260], 2, 2, 16, 16, 200, 8, 3),
       (8, [5000], 2, 1, 3, 64, 4000, 1, 3500), (4, [9000], 3, 3, 1, 100, 7000, 390, 12), (8, [31], 2, 2, 2, 50, 9, 1, 3),
       (8, [400, 30], 3, 3, 17, 5, 300, 1, 90), (4, [5000], 8, 1, 4, 0, 4800, 1, 4000), (8, [300], 5, 1, 5, 9, 200, 16, 5)]
MANY = [(8, [300], 2, 2, 300, 0, 300, 1, 300), (4, [300], 2, 2, 300, 5, 290, 1, 64), (8, [700, 650], 4, 1, 130, 3, 700, 1, 500),
        (4, [513, 0, 1], 2, 1, 17, 16, 256, 1, 200), (8, [1000], 1, 1, 520, 100, 600, 100, 4), (4, [1024], 2, 2, 128, 128, 896, 128, 3),
        (8, [640], 3, 3, 33, 0, 640, 1, 1), (4, [2000], 2, 2, 257, 7, 1500, 50, 9), (8, [90], 2, 2, 200, 20, 60, 1, 30),
        (8, [6000], 1, 1, 40, 33, 5000, 1, 4500), (4, [700], 11, 1, 3, 2, 600, 1, 333)]


@pytest.mark.parametrize("case", FEW + MANY)
def test_attend(qwm, case):
    bits, lengths, H, kv, nq, sink, ring, tpf, frames = case
    rng = np.random.default_rng(sum(lengths) + nq)
    ctx = ctx_of(qwm, H)
    win = fill(qwm, ctx, rng, bits, kv, sink, ring, lengths)
    b = len(lengths)
    q = rows(rng, b, H, nq, "token")
    starts = [max(0, L - nq) for L in lengths]
    out = torch.empty(b, H, nq, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(b, H, nq, dtype=torch.float32, device="cuda")
    qwm.qwm_window_attend(ctx, win, q, ints(starts), ints(lengths), tpf, frames, SCALE, out, lse=lse)
    assert qwm.qwm_sync_status(ctx) == 0
    check_attention(win, q, starts, lengths, tpf, frames, SCALE, out, lse)


@pytest.mark.parametrize("nq,q0", [(3, 10_000), (40, 10_000), (2, 0), (70, 0), (2, 95), (64, 70)])
def test_attend_query_positions_away_from_the_end(qwm, nq, q0):
    """Queries past the cached tokens (their window may hold none), at the beginning, and in the middle
    of a cache whose later tokens they must not see."""
    rng = np.random.default_rng(q0 + nq)
    ctx = ctx_of(qwm, 2)
    win = fill(qwm, ctx, rng, 8, 2, 0 if q0 else 6, 120, [130])
    q = rows(rng, 1, 2, nq)
    out = torch.empty(1, 2, nq, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, 2, nq, dtype=torch.float32, device="cuda")
    for tpf, frames in ((1, 50), (16, 2)):
        qwm.qwm_window_attend(ctx, win, q, ints([q0]), ints([130]), tpf, frames, SCALE, out, lse=lse)
        check_attention(win, q, [q0], [130], tpf, frames, SCALE, out, lse)


@pytest.mark.parametrize("nq,g", [(2, 2), (6, 8), (100, 2)])
def test_attend_padded_batch_strides_and_rows_left_alone(qwm, nq, g):
    rng = np.random.default_rng(nq)
    H, kv, lengths, counts = 2 * g, 2, [90, 200, 150, 10], [nq, 0, nq - 1, 1]
    ctx = ctx_of(qwm, H)
    win = fill(qwm, ctx, rng, 4, kv, 3, 160, lengths)
    q = rows(rng, 4, H, nq, "padded")
    q[1] = float("nan")                       # a skipped sequence's rows are not read
    starts = [max(0, lengths[0] - nq), 3, -1, 9]
    big = torch.full((4, nq, H, 136), 5.0, dtype=torch.bfloat16, device="cuda")
    out = big.permute(0, 2, 1, 3)[..., :128]
    lse = torch.full((4, H, nq), 5.0, dtype=torch.float32, device="cuda")
    qwm.qwm_window_attend(ctx, win, q, ints(starts), ints(lengths), 1, 100, SCALE, out, lse=lse, q_count=ints(counts, torch.int32))
    assert qwm.qwm_sync_status(ctx) == 0
    check_attention(win, q, starts, lengths, 1, 100, SCALE, out, lse, counts=counts)
    assert bool((big[..., 128:] == 5).all())
    for i, c in ((1, 0), (2, 0), (3, 1)):
        assert bool((out[i][:, c:] == 5).all()) and bool((lse[i][:, c:] == 5).all())


@pytest.mark.parametrize("nq", [1, 12, 40, 300])
def test_attend_fp32_and_merge(qwm, nq):
    """Two windows over different tokens merged equal attention over both; a window that shows a row no
    key leaves the row as it was; both empty stay empty."""
    rng = np.random.default_rng(nq)
    H, ctx = 2, ctx_of(qwm, 2)
    a, c = fill(qwm, ctx, rng, 8, 2, 0, 200, [180]), fill(qwm, ctx, rng, 8, 2, 4, 90, [90])
    q = rows(rng, 1, H, nq)
    out = torch.empty(1, H, nq, 128, dtype=torch.float32, device="cuda")
    lse = torch.empty(1, H, nq, dtype=torch.float32, device="cuda")
    qwm.qwm_window_attend(ctx, a, q, ints([10 ** 6]), ints([180]), 10 ** 9, 1, SCALE, out, lse=lse)   # all keys
    check_attention(a, q, [10 ** 6], [180], 10 ** 9, 1, SCALE, out, lse, out_eps=2.0 ** -23)
    alone = (out.clone(), lse.clone())
    qwm.qwm_window_attend(ctx, c, q, ints([10 ** 6]), ints([90]), 10 ** 9, 1, SCALE, out, lse=lse, merge=True)
    for h in range(H):
        pa, ka, va = decoded(a, 0, h, 180)
        pc, kc, vc = decoded(c, 0, h, 90)
        k, v = np.concatenate([ka, kc]), np.concatenate([va, vc])
        want, wl, mag, spread = ref.attend(f64(q[0, h]), k, v, np.zeros(len(k), np.int64), 0, 10 ** 9, 1, 0, SCALE)
        eps = (2.0 ** -11 + 2.0 ** -16 * mag + 2.0 ** -20)[:, None]
        # the parts' weights add two exp2 and one division of fp32 each
        assert np.all(np.abs(f64(out[0, h]) - want) <= 2 * (eps + 2.0 ** -20) * spread + 300 * 2.0 ** -25 * np.abs(v).max())
        assert np.all(np.abs(lse[0, h].double().cpu().numpy() - wl) <= 2.0 ** -16 * mag + 2.0 ** -19 + 2.0 ** -21 * np.abs(wl))
    out.copy_(alone[0]), lse.copy_(alone[1])
    empty = qwm.Window.empty(8, 1, 2, 0, 50)
    qwm.qwm_window_attend(ctx, empty, q, ints([5]), ints([0]), 1, 10, SCALE, out, lse=lse, merge=True)
    assert torch.equal(out, alone[0]) and torch.equal(lse, alone[1])
    qwm.qwm_window_attend(ctx, empty, q, ints([5]), ints([0]), 1, 10, SCALE, out, lse=lse)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    qwm.qwm_window_attend(ctx, empty, q, ints([5]), ints([0]), 1, 10, SCALE, out, lse=lse, merge=True)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    qwm.qwm_window_attend(ctx, a, q, ints([10 ** 6]), ints([180]), 10 ** 9, 1, SCALE, out, lse=lse, merge=True)
    assert bool(((out - alone[0]).abs() <= 2.0 ** -21 * alone[0].abs()).all()) and bool(((lse - alone[1]).abs() <= 2.0 ** -21 * alone[1].abs() + 2.0 ** -22).all())


@pytest.mark.parametrize("nq", [2, 64])
def test_attend_sharp_and_growing_logits(qwm, nq):
    """Keys that grow along the sequence raise the running maximum again and again; masked keys may be
    the largest."""
    rng = np.random.default_rng(5)
    ctx = ctx_of(qwm, 1)
    win = qwm.Window.empty(8, 1, 1, 2, 600)
    k, v = rows(rng, 1, 1, 600, outliers=False), rows(rng, 1, 1, 600)
    k *= torch.linspace(0.01, 30, 600, device="cuda")[None, None, :, None]
    qwm.qwm_window_write(ctx, win, k, v, ints([0]))
    q = rows(rng, 1, 1, nq, scale=3.0, outliers=False)
    out = torch.empty(1, 1, nq, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, 1, nq, dtype=torch.float32, device="cuda")
    for q0, frames in ((600 - nq, 600), (300, 200)):
        qwm.qwm_window_attend(ctx, win, q, ints([q0]), ints([600]), 1, frames, SCALE, out, lse=lse)
        check_attention(win, q, [q0], [600], 1, frames, SCALE, out, lse)


@pytest.mark.parametrize("nq", [1, 33])
def test_attend_query_range_error(qwm, nq):
    rng = np.random.default_rng(1)
    ctx = ctx_of(qwm, 1)
    win = fill(qwm, ctx, rng, 8, 1, 0, 40, [40])
    q = rows(rng, 1, 1, nq)
    q[0, 0, 0, 5] = 1e5
    out = torch.empty(1, 1, nq, 128, dtype=torch.bfloat16, device="cuda")
    qwm.qwm_window_attend(ctx, win, q, ints([40]), ints([40]), 1, 50, SCALE, out)
    assert qwm.qwm_sync_status(ctx) == qwm.QWM_ERR_RANGE and qwm.qwm_sync_status(ctx) == 0


def test_split_parts_do_not_depend_on_the_run(qwm):
    """The same call gives the same bits every time (no order of arrival in any sum)."""
    rng = np.random.default_rng(2)
    ctx = ctx_of(qwm, 4)
    for nq, n in ((1, 6000), (1, 12000), (30, 6000)):
        win = fill(qwm, ctx, rng, 4, 2, 4, n, [n])
        q = rows(rng, 1, 4, nq)
        got = []
        for _ in range(3):
            out = torch.empty(1, 4, nq, 128, dtype=torch.float32, device="cuda")
            lse = torch.empty(1, 4, nq, dtype=torch.float32, device="cuda")
            qwm.qwm_window_attend(ctx, win, q, ints([n - 10]), ints([n]), 1, n, SCALE, out, lse=lse)
            got.append((out, lse))
        if (nq, n) != (1, 6000):   # parts joined through the workspace; the first inside a cluster
            assert qwm.qwm_window_attend_workspace(ctx, win, nq, 1, n) > 0
        for o, s in got[1:]:
            assert torch.equal(o, got[0][0]) and torch.equal(s, got[0][1])


# ------------------------------------------------------------------ together

def test_generation_captured_in_a_graph(qwm):
    """Turn, write and attend one token at a time, the step captured once and replayed with positions
    advanced on the device, on a stream of its own; equals the eager run bit for bit, and the reference."""
    rng = np.random.default_rng(8)
    H, kv, T = 4, 2, 40
    ctx, spec = ctx_of(qwm, H), qwm.RopeSpec((64, 32, 32), grid=(3, 4), pairing="half")
    qs, ks, vs = rows(rng, T, H, 1, "head"), rows(rng, T, kv, 1, "head"), rows(rng, T, kv, 1, "head")

    def make():
        s = dict(win=qwm.Window.empty(8, 1, kv, 3, 16), q=torch.empty_like(qs[:1]), k=torch.empty_like(ks[:1]), v=torch.empty_like(vs[:1]),
                 pos=ints([0]), len=ints([1]), out=torch.empty(1, H, 1, 128, dtype=torch.bfloat16, device="cuda"),
                 lse=torch.empty(1, H, 1, dtype=torch.float32, device="cuda"))
        return s

    def step(s):
        turned = torch.empty_like(s["q"])
        qwm.qwm_rope(ctx, spec, s["q"], s["pos"], turned)
        qwm.qwm_window_write(ctx, s["win"], s["k"], s["v"], s["pos"], rope=spec)
        qwm.qwm_window_attend(ctx, s["win"], turned, s["pos"], s["len"], 1, 12, SCALE, s["out"], lse=s["lse"])
        s["pos"] += 1
        s["len"] += 1
        s["turned"] = turned

    eager, graphed = make(), make()
    for s in (eager, graphed):
        s["q"].copy_(qs[:1]), s["k"].copy_(ks[:1]), s["v"].copy_(vs[:1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step(graphed)   # once outside, as any capture wants
        graphed["pos"].zero_(), graphed["len"].fill_(1)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step(graphed)
    torch.cuda.current_stream().wait_stream(side)
    for t in range(T):
        for s in (eager, graphed):
            s["q"].copy_(qs[t:t + 1]), s["k"].copy_(ks[t:t + 1]), s["v"].copy_(vs[t:t + 1])
        step(eager)
        graph.replay()
        assert torch.equal(eager["out"], graphed["out"]) and torch.equal(eager["lse"], graphed["lse"])
        check_attention(eager["win"], eager["turned"], [t], [t + 1], 1, 12, SCALE, eager["out"], eager["lse"])
    assert torch.equal(eager["win"].k_codes, graphed["win"].k_codes)


def test_two_calls_at_once(qwm):
    """Split calls on two streams, each with its own workspace, do not disturb one another."""
    rng = np.random.default_rng(12)
    ctx = ctx_of(qwm, 2)
    win = fill(qwm, ctx, rng, 8, 2, 0, 9000, [9000])
    qa, qb = rows(rng, 1, 2, 1), rows(rng, 1, 2, 30)
    want = []
    for q in (qa, qb):
        out = torch.empty(1, 2, q.shape[2], 128, dtype=torch.float32, device="cuda")
        qwm.qwm_window_attend(ctx, win, q, ints([8999]), ints([9000]), 1, 9000, SCALE, out)
        want.append(out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    q0, ln = ints([8999]), ints([9000])
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for s, q, g in zip(streams, (qa, qb), got):
            with torch.cuda.stream(s):
                out = torch.empty(1, 2, q.shape[2], 128, dtype=torch.float32, device="cuda")
            qwm.qwm_window_attend(ctx, win, q, q0, ln, 1, 9000, SCALE, out, stream=s)
            g.append(out)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, o) for o in g)


@pytest.mark.parametrize("bits,tpf,rope", [(8, None, True), (4, 64, False)])
def test_windowed_layer_over_a_packed_history(qwm, bits, tpf, rope):
    """A stream of chunks: the newest two in the window, older ones read back and packed to 2 bits.  The
    output equals 64-bit attention over the packed chunks (the oracle's) and the window's values joined by
    their log-sum-exps, within the attention's bar of 2e-2 x RMS(O)."""
    import oracle
    import synth
    from bit_kv_cache_qsac_gb300 import stream
    from helpers import chunk_head, from_u16, to_u16
    H, n = 2, 256
    ctx = qwm.Context(heads=H, n_centroids=64)
    spec = qwm.RopeSpec((44, 42, 42), grid=(16, 16)) if rope else None
    layer = stream.WindowedLayer(ctx, n, 2, bits=bits, tpf=tpf, rope=spec)
    keys, vals = synth.keys(synth.TINY), synth.values(synth.TINY)
    for t in range(4):
        k, v = (from_u16(np.ascontiguousarray(x[:, t * n:(t + 1) * n]), torch.bfloat16) for x in (keys, vals))
        q = from_u16(synth.queries(synth.TINY, t, n), torch.bfloat16)
        out = layer.step(k, v, q)
        assert layer.check() == 0
        assert len(layer.packed.chunks) == max(0, t - 1)
        if rope:
            turned = torch.empty(1, H, n, 128, dtype=torch.bfloat16, device="cuda")
            qwm.qwm_rope(ctx, spec, q[None], ints([t * n]), turned)
            q = turned[0]
        length = (t + 1) * n
        for h in range(H):
            pos, kw, vw = decoded(layer.window, 0, h, length)
            assert pos[0] == max(0, length - 2 * n)
            want, lse, _, _ = ref.attend(f64(q[h]), kw, vw, pos, t * n, tpf or n, 10 ** 6, 0, SCALE)
            if layer.packed.chunks:
                heads = [chunk_head(c, h) for c in layer.packed.chunks]
                far, far_lse = oracle.attend_rows(to_u16(q[h]), np.arange(n), heads, SCALE, with_lse=True)
                top = np.maximum(lse, far_lse)
                a, b = np.exp2(lse - top)[:, None], np.exp2(far_lse - top)[:, None]
                want = (a * want + b * far) / (a + b)
            err = np.abs(f64(out[h]) - want).max() / np.sqrt(np.mean(want ** 2))
            assert err <= 2e-2, (t, h, err)
    with pytest.raises(ValueError):
        layer.step(k[:, :10], v[:, :10], q[:, :10])


# (bits, batch, H, kv, nq, counts, sink, ring, length, tpf, frames): more units of 512 rows than the GPU holds at
# once, so that a pair of CTAs walks over several, of one and of two Query tiles, with and without live rows
UNITS = [(4, 2, 48, 48, 530, None, 5, 600, 700, 1, 300), (4, 7, 24, 12, 300, [300, 0, 10, 131, 300, 256, 257], 0, 900, 900, 64, 4),
         (4, 40, 8, 4, 40, None, 3, 200, 190, 1, 60), (4, 1, 90, 90, 1100, None, 0, 64, 1500, 1, 20)]


@pytest.mark.parametrize("case", UNITS)
def test_attend_many_units(qwm, case):
    bits, b, H, kv, nq, counts, sink, ring, length, tpf, frames = case
    rng = np.random.default_rng(nq)
    ctx = ctx_of(qwm, H)
    win = fill(qwm, ctx, rng, bits, kv, sink, ring, [length - 3 * i for i in range(b)])
    lengths = [length - 3 * i for i in range(b)]
    starts = [max(0, n - nq) for n in lengths]
    q = rows(rng, b, H, nq)
    out = torch.full((b, H, nq, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b, H, nq), 5.0, dtype=torch.float32, device="cuda")
    for _ in range(2):
        qwm.qwm_window_attend(ctx, win, q, ints(starts), ints(lengths), tpf, frames, SCALE, out, lse=lse,
                              q_count=ints(counts, torch.int32) if counts else None)
    assert qwm.qwm_sync_status(ctx) == 0
    slots = sink + ring
    values = torch.empty(2, b, kv, slots, 128, dtype=torch.bfloat16, device="cuda")   # 4-bit values are exact in bf16
    ahead = torch.full((b, slots), -1, dtype=torch.int64)
    for i, n in enumerate(lengths):
        pos = ref.held(n, sink, ring)
        ahead[i, :len(pos)] = torch.tensor(pos)
    for i in range(b):   # held tokens: the sinks, then the last ring ones
        m = int((ahead[i] >= 0).sum())
        head = min(sink, m)
        one = qwm.Window(bits, sink, ring, *(t[i:i + 1] for t in (win.k_codes, win.k_step, win.v_codes, win.v_step)))
        for at, cnt in ((0, head), (head, m - head)):
            if cnt:
                kh, vh = (torch.empty(1, kv, cnt, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
                qwm.qwm_window_read(ctx, one, ints([int(ahead[i, at])]), ints([lengths[i]]), kh, vh)
                values[0, i, :, at:at + cnt], values[1, i, :, at:at + cnt] = kh[0], vh[0]
    for i in range(b):
        live = counts[i] if counts else nq
        assert bool((out[i][:, live:] == 5).all()) and bool((lse[i][:, live:] == 5).all())
        if not live:
            continue
        pos = ahead[i][ahead[i] >= 0].cuda()
        k, v = (values[e, i, :, :pos.numel()].double().repeat_interleave(H // kv, 0) for e in range(2))
        fq = (torch.arange(live, device="cuda") + starts[i]) // tpf
        see = (pos // tpf <= fq[:, None]) & ((fq[:, None] - pos // tpf < frames) | (pos < sink))
        qq = q[i, :, :live].double()
        x = (qq @ k.transpose(1, 2) * (SCALE * math.log2(math.e))).masked_fill(~see, -math.inf)
        wl = torch.logsumexp(x * math.log(2.0), -1) / math.log(2.0)
        w = torch.exp2(x - wl[..., None])
        want, spread = w @ v, w @ v.abs()
        mag = (qq.abs() @ k.abs().transpose(1, 2)).amax(-1) * SCALE * math.log2(math.e)
        eps = (2.0 ** -11 + 2.0 ** -16 * mag + 2.0 ** -20)[..., None]
        bound = 2 * eps * spread + pos.numel() * 2.0 ** -25 * v.abs().max() + 2.0 ** -8 * want.abs()
        some = see.any(1)
        assert bool((out[i][:, :live][:, ~some] == 0).all()) and bool(torch.isneginf(lse[i][:, :live][:, ~some]).all())
        assert bool(((out[i, :, :live].double() - want).abs() <= bound)[:, some].all()), i
        off = (lse[i, :, :live].double() - wl).abs() <= 2.0 ** -16 * mag + 2.0 ** -20 + 2.0 ** -22 * wl.abs()
        assert bool(off[:, some].all()), i


# ------------------------------------------------------------------ values only the device sees

FAR = [2 ** 63 - 1, 2 ** 62 + 1, -2 ** 63, -1]   # no position of a token: the sequence is skipped


@pytest.mark.parametrize("bits", [8, 4])
def test_positions_outside_the_range_leave_everything_as_it_was(qwm, bits):
    rng = np.random.default_rng(21)
    b, n, ctx = len(FAR), 9, ctx_of(qwm, 2)
    x = rows(rng, b, 2, n)
    five = torch.full_like(x, 5.0)
    out = five.clone()
    qwm.qwm_rope(ctx, qwm.RopeSpec((64, 32, 32)), x, ints(FAR), out)
    assert torch.equal(out, five)
    win = qwm.Window.empty(bits, b, 2, 4, 60)
    for spec in (None, qwm.RopeSpec((64, 32, 32)), qwm.RopeSpec((128, 0, 0), pairing="half")):
        qwm.qwm_window_write(ctx, win, x, x, ints(FAR), rope=spec)
    assert not any(bool(t.any()) for t in (win.k_codes, win.k_step, win.v_codes, win.v_step))
    kh, vh = torch.full((b, 2, n, 128), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((b, 2, n, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    qwm.qwm_window_read(ctx, win, ints(FAR), ints([64] * b), kh, vh)
    assert bool((kh == 5).all()) and bool((vh == 5).all())
    for nq in (1, 40):
        q = rows(rng, b, 2, nq)
        o = torch.full((b, 2, nq, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((b, 2, nq), 5.0, dtype=torch.float32, device="cuda")
        qwm.qwm_window_attend(ctx, win, q, ints(FAR), ints([64] * b), 1, 60, SCALE, o, lse=lse)
        assert bool((o == 5).all()) and bool((lse == 5).all())


@pytest.mark.parametrize("nq", [1, 12, 40, 300])
@pytest.mark.parametrize("ring", [60, 9000])   # 9000: the keys are split
def test_negative_lengths_hold_no_token(qwm, nq, ring):
    rng = np.random.default_rng(22)
    lengths, ctx = [-1, -5000, -2 ** 40, -2 ** 63], ctx_of(qwm, 2)
    b, win = len(lengths), qwm.Window.empty(8, len(lengths), 1, 4, ring)
    win.k_codes.fill_(200), win.v_codes.fill_(200), win.k_step.fill_(0x78), win.v_step.fill_(0x78)
    q = rows(rng, b, 2, nq)
    out = torch.full((b, 2, nq, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b, 2, nq), 5.0, dtype=torch.float32, device="cuda")
    qwm.qwm_window_attend(ctx, win, q, ints([100] * b), ints(lengths), 1, ring, SCALE, out, lse=lse)
    assert qwm.qwm_sync_status(ctx) == 0
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    kh = torch.full((b, 1, 7, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    qwm.qwm_window_read(ctx, win, ints([0, 2, 3, 4]), ints(lengths), kh, None)
    assert bool((kh == 0).all())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("length", [1, 63, 64, 65, 128, 129, 193, 700])   # halves of a stage, stages, more than the stages
@pytest.mark.parametrize("nq", [33, 256, 257])                           # one Query tile and just past it
def test_attend_around_one_query_tile(qwm, bits, length, nq):
    rng = np.random.default_rng(length + nq)
    ctx = ctx_of(qwm, 1)
    win = fill(qwm, ctx, rng, bits, 1, 2, 800, [length])
    q = rows(rng, 1, 1, nq)
    out = torch.empty(1, 1, nq, 128, dtype=torch.float32, device="cuda")
    lse = torch.empty(1, 1, nq, dtype=torch.float32, device="cuda")
    q0 = max(0, length - nq)
    for tpf, frames in ((1, 800), (1, 50), (100, 2)):
        qwm.qwm_window_attend(ctx, win, q, ints([q0]), ints([length]), tpf, frames, SCALE, out, lse=lse)
        assert qwm.qwm_sync_status(ctx) == 0
        check_attention(win, q, [q0], [length], tpf, frames, SCALE, out, lse, out_eps=2.0 ** -22)
