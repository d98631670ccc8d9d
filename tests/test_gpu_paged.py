"""The paged operators on the GPU against the 64-bit reference: norms with the rotation, page tables and
slot maps, the paged cache (written and read back), attention of packed batches, and runs of them
together."""
import math

import numpy as np
import pytest

import paged_ref
import window_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)
PAGES = [16, 32, 64, 128, 256]


@pytest.fixture(scope="module")
def qwm():
    import bit_kv_cache_qsac_gb300 as q
    return q


_CTX = {}


def ctx_of(qwm, heads):
    if heads not in _CTX:
        _CTX[heads] = qwm.Context(heads=heads)
    return _CTX[heads]


def rows(rng, h, n, layout="token", scale=1.0, outliers=True):
    """bf16 activations [h][n][128]: token-major, head-major or padded memory."""
    x = rng.standard_normal((h, n, 128)).astype(np.float32) * scale
    if outliers:
        x[..., rng.permutation(128)[:8]] *= 4
    t = torch.from_numpy(x).to(torch.bfloat16).cuda()
    if layout == "token":
        t = t.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    elif layout == "padded":
        big = torch.full((h, n, 160), 9.0, dtype=torch.bfloat16, device="cuda")
        big[..., :128] = t
        t = big[..., :128]
    return t


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def ints(v, dtype=torch.int64):
    return v if isinstance(v, torch.Tensor) else torch.tensor(v, dtype=dtype, device="cuda")


def status(qwm, ctx):
    """The recorded error, which this clears."""
    try:
        return qwm.qwm_sync_status(ctx)
    except qwm.QwmError as e:
        return e.status


# ------------------------------------------------------------------ norm and rotation

SPECS = {"video": dict(dims=(44, 42, 42), theta=10000.0, pairing="interleaved", grid=(45, 80)),
         "text": dict(dims=(128, 0, 0), theta=1e6, pairing="half"),
         "shared": dict(dims=(32, 48, 48), theta=(1e4, 1e3, 50.0), pairing="half", shared_freq=True, grid=(7, 3)),
         "partial": dict(dims=(16, 0, 16), theta=256.0, pairing="half", grid=(2, 9)),
         "odd": dict(dims=(2, 4, 30), theta=100.0, pairing="interleaved", grid=(5, 5)),
         "none": None}


def turned(y, kw, pos):
    th = kw.get("theta", 10000.0)
    return ref.rope(y, kw["dims"], th if isinstance(th, tuple) else (th,) * 3, kw["pairing"], kw.get("shared_freq", False), pos)


def norm_bound(y, want, kw):
    """fp32 throughout: the sum of squares carries 13 roundings, half of which reach the root, the root, the
    quotient and the two products one each (10 x 2^-24); cosine and sine within 2^-24, the two products and the
    sum another three: under 2^-20 of |a| + |b|; then rounded to bf16 (2^-8 relative)."""
    pair = np.abs(y).copy()
    if kw:
        half = sum(kw["dims"]) // 2
        for i in range(half):
            c = (2 * i, 2 * i + 1) if kw["pairing"] == "interleaved" else (i, i + half)
            pair[..., c[0]] = pair[..., c[1]] = np.abs(y[..., c[0]]) + np.abs(y[..., c[1]])
    return 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * pair


@pytest.mark.parametrize("name", SPECS)
@pytest.mark.parametrize("b,h,n,layout,start,weights", [(1, 3, 1, "token", 0, "one"), (2, 5, 37, "head", 1000, "heads"),
                                                        (3, 1, 16, "padded", 3_000_000_000, None), (1, 40, 65, "token", 75_600, "heads")])
def test_norm_rope(qwm, name, b, h, n, layout, start, weights):
    kw = SPECS[name]
    rng = np.random.default_rng(b * 100 + n)
    x = torch.stack([rows(rng, h, n, layout) for _ in range(b)]) if layout != "padded" else rows(rng, b * h, n, "padded").unflatten(0, (b, h))
    w = torch.from_numpy(rng.uniform(0.2, 2.0, (h, 128) if weights == "heads" else (128,)).astype(np.float32)).cuda() if weights else None
    starts = [start + 11 * i for i in range(b)]
    out = torch.empty(b, h, n, 128, dtype=torch.bfloat16, device="cuda")
    spec = qwm.RopeSpec(**kw) if kw else None
    qwm.qwm_norm_rope(ctx_of(qwm, h), spec, x, w, 1e-6, out, start=ints(starts) if kw else None)
    xr, got = f64(x), f64(out)
    for i in range(b):
        pos = ref.grid_positions(starts[i], n, *(kw or {}).get("grid", (1, 1)))
        for j in range(h):
            g = f64(w[j] if weights == "heads" else w) if weights else np.ones(128)
            y = paged_ref.norm(xr[i, j], g, 1e-6)
            want = turned(y, kw, pos) if kw else y
            assert np.all(np.abs(got[i, j] - want) <= norm_bound(y, want, kw)), (i, j)
    at = ints([[s + k for k in range(n)] for s in starts])
    again = torch.empty_like(out)
    qwm.qwm_norm_rope(ctx_of(qwm, h), spec, x, w, 1e-6, again, at=at)
    assert torch.equal(out, again)


@pytest.mark.parametrize("name", ["video", "shared"])
def test_norm_rope_in_place_given_positions_and_skipped_rows(qwm, name):
    kw, rng = SPECS[name], np.random.default_rng(7)
    x = rows(rng, 4, 21)[None]
    keep = x.clone()
    pos = ints(rng.integers(-(2 ** 31), 2 ** 31, (1, 21, 3)).tolist(), torch.int32)
    at = ints([[-1 if i in (0, 5, 20) else (2 ** 62 + 1 if i == 9 else i) for i in range(21)]])
    qwm.qwm_norm_rope(ctx_of(qwm, 4), qwm.RopeSpec(**kw), x, None, 0.0, x, at=at, pos=pos)
    left = [0, 5, 9, 20]
    assert torch.equal(x[:, :, left], keep[:, :, left])
    live = [i for i in range(21) if i not in left]
    for j in range(4):
        y = paged_ref.norm(f64(keep[0, j, live]), 1.0, 0.0)
        want = turned(y, kw, pos[0, live].cpu().numpy().astype(np.int64))
        assert np.all(np.abs(f64(x[0, j, live]) - want) <= norm_bound(y, want, kw))


@pytest.mark.parametrize("name", ["none", "text", "video"])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30])
def test_norm_rope_rows_beyond_the_range_of_squares(qwm, name, eps):
    """Magnitudes whose squares overflow or vanish in fp32, beside ordinary rows, zeros, infinities and NaN."""
    kw, rng = SPECS[name], np.random.default_rng(3)
    scale = 2.0 ** np.array([0, 100, 126, 64, -60, -70, -100, -120, 0, 0, 0, 0])
    x = rows(rng, 2, 12, outliers=False).double() * torch.from_numpy(scale).cuda()[None, :, None]
    x = x.clamp(-2.0 ** 127, 2.0 ** 127).to(torch.bfloat16)
    x[:, 9] = 0.0
    x[:, 10, 17] = math.inf
    x[:, 11, 40] = math.nan
    out = torch.empty(1, 2, 12, 128, dtype=torch.bfloat16, device="cuda")
    qwm.qwm_norm_rope(ctx_of(qwm, 2), qwm.RopeSpec(**kw) if kw else None, x[None], None, eps, out, start=ints([5]) if kw else None)
    pos = ref.grid_positions(5, 12, *(kw or {}).get("grid", (1, 1)))
    for j in range(2):
        y = paged_ref.norm(f64(x[j]), 1.0, float(np.float32(eps)))
        y[10][np.arange(128) != 17] = 0.0   # finite over infinite
        want = turned(y, kw, pos) if kw else y
        got = f64(out[0, j])
        nan = np.isnan(want)
        assert np.array_equal(nan, np.isnan(got)), np.argwhere(nan != np.isnan(got))[:5]
        # results below the normal numbers keep fp32's grid of 2^-149, 2^-133 in bf16
        assert np.all((np.abs(got - want) <= norm_bound(y, want, kw) + 2.0 ** -133)[~nan])


def test_norm_without_positions_is_the_norm_and_rope_of_ones_is_rope_of_the_normed(qwm):
    rng = np.random.default_rng(1)
    ctx, x = ctx_of(qwm, 3), rows(rng, 3, 40)[None]
    plain, turned_ = (torch.empty(1, 3, 40, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qwm.qwm_norm_rope(ctx, None, x, None, 1e-5, plain)
    qwm.qwm_norm_rope(ctx, qwm.RopeSpec((0, 0, 0)), x, None, 1e-5, turned_, start=ints([9]))
    assert torch.equal(plain, turned_)


# ------------------------------------------------------------------ page tables


class Both:
    """A page table on the device beside the reference's."""

    def __init__(self, qwm, batch, width, page, pages):
        self.qwm, self.ctx = qwm, ctx_of(qwm, 1)
        self.ref = paged_ref.Pages(batch, width, page, pages)
        self.tab = qwm.PageTable.empty(batch, width, page, pages)

    def update(self, keep, count, n):
        b = self.tab.batch
        dev = dict(keep=ints(keep) if keep is not None else None, count=ints(count, torch.int32) if count is not None else None)
        if count is not None:
            dev.update(first=torch.full((b,), 7, dtype=torch.int32, device="cuda"), granted=torch.full((b,), 7, dtype=torch.int32, device="cuda"),
                       slot=torch.full((n,), 7, dtype=torch.int64, device="cuda"), at=torch.full((n,), 7, dtype=torch.int64, device="cuda"))
        self.qwm.qwm_pages_update(self.ctx, self.tab, **dev)
        first, granted, slot, at = self.ref.update(keep, count, n)
        if count is not None:
            for name, want in (("first", first), ("granted", granted), ("slot", slot), ("at", at)):
                assert dev[name].tolist() == want, name
        self.check()
        return dev

    def check(self):
        assert self.tab.length.tolist() == self.ref.length
        assert np.array_equal(self.tab.table.cpu().numpy(), self.ref.table())
        assert int(self.tab.free_count) == len(self.ref.free)
        assert np.array_equal(self.tab.free.cpu().numpy(), self.ref.stack())


@pytest.mark.parametrize("batch,width,page,pages,most", [(1, 3, 16, 3, 20), (5, 9, 16, 30, 60), (64, 20, 64, 700, 300), (300, 6, 256, 900, 700),
                                                         (1025, 4, 32, 2000, 40), (4096, 3, 16, 5000, 30)])
def test_pages_update(qwm, batch, width, page, pages, most):
    rng = np.random.default_rng(batch)
    both = Both(qwm, batch, width, page, pages)
    for step in range(6):
        keep = None if step == 0 else [int(rng.choice([0, max(0, L - rng.integers(0, 5)), L + 3, -4])) if rng.random() < 0.5 else L
                                       for L in both.ref.length]
        count = None if step == 3 else [int(rng.choice([0, 1, rng.integers(0, most + 1), -2, 1])) for _ in range(batch)]
        n = 0 if count is None else max(0, sum(max(0, c) for c in count) + int(rng.choice([0, 9, -most // 2])))
        both.update(keep, count, n)
    assert status(qwm, both.ctx) == qwm.QWM_OK


def test_pages_refusals_in_the_batch(qwm):
    both = Both(qwm, 6, 4, 16, 8)
    assert both.update(None, [30, 0, 65, 17, 5, 20], 200)["granted"].tolist() == [30, 0, 0, 17, 5, 20]   # 65 passes the width
    # one page left of 8; the first needs two, those behind it that need one are refused with it, who needs none is not
    dev = both.update(None, [20, 3, 0, 1, 11, 1], 100)
    assert dev["granted"].tolist() == [0, 0, 0, 1, 11, 1]
    # rows that pass n, also beyond 2^31
    dev = both.update([0] * 6, [2 ** 31 - 1, 5, 2 ** 31 - 1, 5, 0, 1], 10)
    assert dev["granted"].tolist() == [0] * 6
    assert both.update(None, [4, 7, 3, 2, 0, 1], 8)["granted"].tolist() == [4, 0, 0, 0, 0, 0]
    both.update([2] + [0] * 5, None, 0)


def test_pages_shrinking_and_growing_again_gives_the_same_pages(qwm):
    both = Both(qwm, 3, 8, 16, 20)
    both.update(None, [100, 20, 50], 170)
    table = both.tab.table.clone()
    both.update([16, 0, 33], [84, 20, 17], 200)
    assert torch.equal(both.tab.table, table)
    qwm.qwm_pages_reset(both.ctx, both.tab)
    both.ref = paged_ref.Pages(3, 8, 16, 20)
    both.check()


def test_pages_lengths_outside_the_table_are_recorded(qwm):
    tab, ctx = qwm.PageTable.empty(2, 4, 16, 8), ctx_of(qwm, 1)
    tab.length.copy_(ints([-5, 3]))
    out = dict(first=ints([0, 0], torch.int32), granted=ints([0, 0], torch.int32), slot=ints([0] * 4), at=ints([0] * 4))
    qwm.qwm_pages_update(ctx, tab, count=ints([2, 1], torch.int32), **out)
    assert status(qwm, ctx) == qwm.QWM_ERR_RANGE
    assert out["at"].tolist() == [0, 1, 3, -1] and tab.length.tolist() == [2, 4]


# ------------------------------------------------------------------ the paged cache


def slots_of(rng, n, page, pages):
    """Distinct slots of scattered pages."""
    order = rng.permutation(pages)
    return [int(order[i // page]) * page + i % page for i in range(n)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("name,norm", [(None, False), ("text", "one"), ("video", "heads"), (None, "one"), ("partial", False)])
def test_write_and_read_back(qwm, bits, page, name, norm):
    """The codes of normed and turned Keys are those of qwm_norm_rope's (qwm_rope's) output, bit for bit."""
    rng = np.random.default_rng(page + bits)
    h, n = 3, 77
    pages = -(-n // page) + 3
    ctx, kw = ctx_of(qwm, h), SPECS[name] if name else None
    k, v = rows(rng, h, n), rows(rng, h, n, "padded")
    slot = slots_of(rng, n, page, pages)
    skipped = {3, 40, 76}
    slot = [-1 if i in skipped else s for i, s in enumerate(slot)]
    at = [1000 + 3 * i for i in range(n)]
    if kw:
        at[11] = -1   # a bad position: skipped too
    spec = qwm.RopeSpec(**kw) if kw else None
    w = torch.from_numpy(rng.uniform(0.5, 1.5, (h, 128) if norm == "heads" else (128,)).astype(np.float32)).cuda() if norm else None
    pool = qwm.PagePool.empty(bits, page, pages, h)
    for t in (pool.k_codes, pool.k_step, pool.v_codes, pool.v_step):
        t.fill_(0x33)
    qwm.qwm_paged_write(ctx, pool, k, v, ints(slot), at=ints(at) if kw else None, rope=spec, weight=w, eps=1e-6)
    if kw:
        slot[11] = -1
    ready = k[None].clone()
    if norm:
        qwm.qwm_norm_rope(ctx, spec, k[None], w, 1e-6, ready, at=ints([at]) if kw else None)
    elif kw:
        for i in range(n):
            if at[i] >= 0:
                one = ready[:, :, i:i + 1]
                qwm.qwm_rope(ctx, spec, one, ints([at[i]]), one)
    hats = [torch.full((h, n, 128), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    qwm.qwm_paged_read(ctx, pool, ints(slot), *hats)
    for x, codes, step, hat in ((f64(ready[0]), pool.k_codes, pool.k_step, hats[0]), (f64(v), pool.v_codes, pool.v_step, hats[1])):
        c, s = codes.cpu().numpy(), step.cpu().numpy()
        for j in range(h):
            q, st = ref.quantise(x[j], bits)
            val = ref.bf16(ref.values(ref.pack(q, bits), st, bits))
            for i in range(n):
                if slot[i] < 0:
                    assert not hat[j, i].any()
                    continue
                at_ = (slot[i] // page, j, slot[i] % page)
                assert np.array_equal(c[at_], ref.pack(q, bits)[i]) and np.array_equal(s[at_], st[i])
                assert np.array_equal(f64(hat[j, i]), val[i])
        written = np.zeros(c.shape[:3], bool)
        for s_ in slot:
            if s_ >= 0:
                written[s_ // page, :, s_ % page] = True
        assert np.all(c[~written] == 0x33) and np.all(s[~written] == 0x33)
    only = torch.empty_like(hats[1])
    qwm.qwm_paged_read(ctx, pool, ints(slot), None, only)
    assert torch.equal(only, hats[1])


def test_slots_beyond_the_pool_are_recorded(qwm):
    ctx, pool = ctx_of(qwm, 2), qwm.PagePool.empty(8, 16, 2, 2)
    k = rows(np.random.default_rng(0), 2, 3)
    qwm.qwm_paged_write(ctx, pool, k, k, ints([5, 32, 2 ** 62]))
    assert status(qwm, ctx) == qwm.QWM_ERR_RANGE
    assert int((pool.k_step != 0).any(-1).sum()) == 2   # token 0 of two heads
    hat = torch.full((2, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    qwm.qwm_paged_read(ctx, pool, ints([32, 5]), hat, None)
    assert status(qwm, ctx) == qwm.QWM_ERR_RANGE
    assert not hat[:, 0].any() and hat[:, 1].any()


# ------------------------------------------------------------------ attention


class Batch:
    """Sequences with written tokens, and what their cache stands for."""

    def __init__(self, qwm, rng, bits, page, kv, lengths, spare=3, k_scale=1.0):
        self.qwm, self.page, self.lengths = qwm, page, lengths
        self.ctx = ctx_of(qwm, kv)
        width = max(1, -(-max(lengths) // page))
        need = sum(-(-n // page) for n in lengths)
        self.tab = qwm.PageTable.empty(len(lengths), width, page, need + spare)
        self.tab.free.copy_(torch.from_numpy(rng.permutation(need + spare).astype(np.int32)).cuda())
        self.pool = qwm.PagePool.empty(bits, page, need + spare, kv)
        # what was never written must not matter: codes and steps of NaN and infinities
        for t in (self.pool.k_codes, self.pool.k_step, self.pool.v_codes, self.pool.v_step):
            t.fill_(0xFF)
        n = sum(lengths)
        b = len(lengths)
        slot, at = (torch.zeros(max(n, 1), dtype=torch.int64, device="cuda") for _ in range(2))
        first, granted = (torch.zeros(b, dtype=torch.int32, device="cuda") for _ in range(2))
        qwm.qwm_pages_update(self.ctx, self.tab, first, granted, slot, at, count=ints(lengths, torch.int32))
        assert granted.tolist() == lengths
        k, v = rows(rng, kv, max(n, 1), scale=k_scale), rows(rng, kv, max(n, 1))
        qwm.qwm_paged_write(self.ctx, self.pool, k, v, slot)
        hats = [torch.empty(kv, max(n, 1), 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        qwm.qwm_paged_read(self.ctx, self.pool, slot, *hats)
        # (bf16 would round 8-bit values: from the codes instead)
        c = {t: getattr(self.pool, t).cpu().numpy() for t in ("k_codes", "k_step", "v_codes", "v_step")}
        s = slot.cpu().numpy()
        take = lambda t, j: c[t][s // page, j, s % page]
        k, v = (np.stack([ref.values(take(x + "_codes", j), take(x + "_step", j), bits) for j in range(kv)]) for x in "kv")
        ends = np.cumsum(lengths)
        self.k = [k[:, e - m:e] for e, m in zip(ends, lengths)]
        self.v = [v[:, e - m:e] for e, m in zip(ends, lengths)]


def check(batch, q, out, lse, first, counts, H, tpf, frames, sink, scale=SCALE, out_eps=2.0 ** -8, parts=0.0):
    """Logits: fp32 sums of 128 products of exact fp16 numbers, next to the fp32 rounding of the scale (2^-16 of the
    largest sum of magnitudes, generously); weights are rounded to fp16 (2^-11) or 2^-32 of the largest; the
    sums' and parts' fp32 roundings are within 2^-20."""
    kv = batch.pool.kv_heads
    for b, c in enumerate(counts):
        n = batch.lengths[b]
        if c <= 0:
            continue
        f = first[b]
        for h in range(H):
            kh, vh = batch.k[b][h // (H // kv)], batch.v[b][h // (H // kv)]
            want, wl, mag, spread = ref.attend(f64(q[h, f:f + c]), kh, vh, np.arange(n), n - c, tpf, frames, sink, scale)
            got, gl = f64(out[h, f:f + c]), lse[h, f:f + c].double().cpu().numpy()
            none = np.isneginf(wl)
            assert np.array_equal(none, np.isneginf(gl)), (b, h)
            assert np.all(got[none] == 0)
            eps = (2.0 ** -11 + 2.0 ** -16 * mag + 2.0 ** -20 + parts)[:, None]
            bound = 2 * eps * spread + n * 2.0 ** -32 * np.abs(vh).max() * 2 + out_eps * np.abs(want)
            assert np.all(np.abs(got - want) <= bound), (b, h, np.max(np.abs(got - want) / bound))
            d = np.abs(gl[~none] - wl[~none])
            assert np.all(d <= 2.0 ** -16 * mag[~none] + 2.0 ** -20 + 2.0 ** -22 * np.abs(wl[~none])), (b, h, d.max())


def starts(counts, gap=0):
    first, row = [], 0
    for c in counts:
        first.append(row)
        row += max(0, c) + gap
    return first, row


# (bits, page, lengths, counts, H, kv, tpf, frames, sink)
ALL = 1 << 30
FEW = [(8, 16, [1], [1], 1, 1, 1, ALL, 0), (4, 16, [1], [1], 2, 1, 1, 1, 5), (8, 64, [200, 0, 17, 150], [1, 0, 1, 1], 8, 2, 1, ALL, 0),
       (4, 32, [300, 64, 17, 150], [5, 3, 5, 1], 6, 2, 1, 120, 3), (8, 256, [40, 41], [7, 7], 4, 4, 1, 10, 8), (4, 128, [500], [1], 16, 1, 1, ALL, 0),
       (8, 16, [500], [1], 15, 1, 1, 77, 7), (4, 16, [260], [16], 2, 2, 8, 3, 16), (8, 64, [5000], [3], 2, 1, 1, 3500, 64),
       (4, 128, [9000], [1], 3, 3, 390, 12, 100), (8, 32, [31], [2], 2, 2, 1, 3, 50), (4, 256, [700, 1000, 3], [2, 2, 2], 12, 4, 1, 600, 0),
       (8, 32, [4097, 129, 128, 127], [1, 1, 1, 1], 8, 8, 1, ALL, 0), (4, 16, [33, 900, 31, 65], [1, 2, 3, 4], 4, 2, 1, 40, 20)]
MANY = [(8, 16, [300], [300], 2, 2, 1, ALL, 0), (4, 32, [300], [300], 2, 2, 1, 64, 5), (8, 64, [700, 650], [130, 40], 4, 1, 1, 500, 3),
        (4, 16, [513, 0, 17], [17, 0, 17], 2, 1, 1, 200, 16), (8, 128, [1000], [520], 1, 1, 100, 4, 100), (4, 256, [1024], [128], 2, 2, 128, 3, 128),
        (8, 16, [640], [33], 3, 3, 1, 1, 0), (4, 64, [2000], [257], 2, 2, 50, 9, 7), (8, 32, [90, 600], [90, 1], 2, 2, 1, 30, 20),
        (8, 64, [6000], [40], 1, 1, 1, 4500, 33), (4, 128, [700], [3], 11, 1, 1, 333, 2), (8, 64, [300, 5, 800, 64], [1, 5, 260, 64], 8, 2, 1, ALL, 0)]


@pytest.mark.parametrize("case", FEW + MANY)
@pytest.mark.parametrize("known", [True, False])
def test_attend(qwm, case, known):
    bits, page, lengths, counts, H, kv, tpf, frames, sink = case
    rng = np.random.default_rng(sum(lengths) + sum(counts))
    batch = Batch(qwm, rng, bits, page, kv, lengths)
    first, n = starts(counts, gap=2)
    q = rows(rng, H, n)
    out = torch.full((n, H, 128), 5.0, dtype=torch.bfloat16, device="cuda").permute(1, 0, 2)
    lse = torch.full((H, n), 5.0, dtype=torch.float32, device="cuda")
    qwm.qwm_paged_attend(ctx_of(qwm, H), batch.pool, batch.tab, q, ints(first, torch.int32), ints(counts, torch.int32), SCALE, out, lse=lse, tpf=tpf,
                         frames=frames, sink=sink, max_count=max(counts) if known else None)
    assert status(qwm, ctx_of(qwm, H)) == qwm.QWM_OK
    check(batch, q, out, lse, first, counts, H, tpf, frames, sink)
    mine = np.zeros(n, bool)
    for f, c in zip(first, counts):
        mine[f:f + c] = True
    left = torch.from_numpy(~mine).cuda()
    assert bool((out[:, left] == 5).all()) and bool((lse[:, left] == 5).all())


def gpu_check(batch, q, out, lse, first, counts, H, tpf=1, frames=ALL, sink=0, out_eps=2.0 ** -8, parts=0.0):
    """check() with the reference on the GPU in 64 bits, for larger calls."""
    kv = batch.pool.kv_heads
    for b, c in enumerate(counts):
        n, f = batch.lengths[b], first[b]
        if c <= 0:
            continue
        k, v = (torch.from_numpy(x[b]).cuda().repeat_interleave(H // kv, 0) for x in (batch.k, batch.v))
        j = torch.arange(n, device="cuda")
        fq = ((torch.arange(c, device="cuda") + n - c) // tpf)[:, None]
        see = (j // tpf <= fq) & ((fq - j // tpf < frames) | (j < sink))
        qq = q[:, f:f + c].double()
        x = (qq @ k.transpose(1, 2) * (SCALE * math.log2(math.e))).masked_fill(~see, -math.inf)
        m = x.amax(-1, keepdim=True)
        w = torch.exp2(x - m)
        wl = (m + torch.log2(w.sum(-1, keepdim=True)))[..., 0]
        w = w / w.sum(-1, keepdim=True)
        want, spread = w @ v, w @ v.abs()
        mag = (qq.abs() @ k.abs().transpose(1, 2)).amax(-1) * SCALE * math.log2(math.e)
        eps = (2.0 ** -11 + 2.0 ** -16 * mag + 2.0 ** -20 + parts)[..., None]
        bound = 2 * eps * spread + n * 2.0 ** -32 * v.abs().max() * 2 + out_eps * want.abs()
        assert bool(((out[:, f:f + c].double() - want).abs() <= bound).all()), b
        d = (lse[:, f:f + c].double() - wl).abs()
        assert bool((d <= 2.0 ** -16 * mag + 2.0 ** -20 + 2.0 ** -22 * wl.abs()).all()), b


def attend(qwm, batch, q, first, counts, H, **kw):
    out = kw.pop("out", None)
    if out is None:
        out = torch.zeros(q.shape[1], H, 128, dtype=kw.pop("dtype", torch.bfloat16), device="cuda").permute(1, 0, 2)
    lse = kw.pop("lse", None)
    if lse is None:
        lse = torch.zeros(H, q.shape[1], dtype=torch.float32, device="cuda")
    qwm.qwm_paged_attend(ctx_of(qwm, H), kw.pop("pool", batch.pool), batch.tab, q, ints(first, torch.int32), ints(counts, torch.int32), SCALE, out, lse=lse,
                         **kw)
    return out, lse


@pytest.mark.parametrize("bits,page,lengths,counts,H,kv", [
    (8, 64, [2000, 1300, 700], [2000, 1300, 700], 8, 2), (4, 16, [9000], [1100], 4, 4), (8, 128, [3000], [40], 40, 1), (4, 64, [2500, 30], [1, 2], 40, 1),
    (8, 16, [150_000], [1], 2, 1), (4, 256, [120_001], [9], 2, 2), (8, 32, [70_000], [65], 4, 2)])
def test_attend_larger(qwm, bits, page, lengths, counts, H, kv):
    """Prompts from nothing, few items over long sequences (joined parts), and more heads than the warp tiles take."""
    rng = np.random.default_rng(H + page)
    batch = Batch(qwm, rng, bits, page, kv, lengths)
    first, n = starts(counts)
    q = rows(rng, H, n)
    out, lse = attend(qwm, batch, q, first, counts, H, max_count=max(counts))
    gpu_check(batch, q, out, lse, first, counts, H)
    for _ in range(2):   # nothing depends on the order in which CTAs run
        again, lse2 = attend(qwm, batch, q, first, counts, H, max_count=max(counts))
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("batch_size", [257, 600])
@pytest.mark.parametrize("chunk", [0, 90])
def test_attend_many_sequences(qwm, batch_size, chunk):
    rng = np.random.default_rng(batch_size + chunk)
    lengths = [int(rng.integers(0, 60)) for _ in range(batch_size)]
    counts = [min(n, int(rng.choice([0, 1, 1, 2]))) for n in lengths]
    for i in (3, 255, batch_size - 1):
        lengths[i] = 300
        counts[i] = chunk or 1
    b = Batch(qwm, rng, 8, 16, 2, lengths)
    first, n = starts(counts, gap=1)
    q = rows(rng, 4, n)
    out, lse = attend(qwm, b, q, first, counts, 4, max_count=max(counts))
    gpu_check(b, q, out, lse, first, counts, 4)


@pytest.mark.parametrize("bits,page,lengths,counts,H,kv", [
    (8, 32, [100, 50, 33], [1, 1, 1], 40, 1),      # a token's rows alone are too many for the few rows' kernel
    (4, 64, [300, 20, 129], [1, 1, 0], 24, 1), (8, 16, [70, 600], [2, 1], 62, 2), (4, 16, [40, 300], [9, 30], 17, 1),
    (8, 64, [500, 64], [1, 3], 600, 1)])           # ... and go over two blocks of rows
def test_attend_wide_groups(qwm, bits, page, lengths, counts, H, kv):
    rng = np.random.default_rng(H + kv)
    b = Batch(qwm, rng, bits, page, kv, lengths)
    first, n = starts(counts, gap=1)
    q = rows(rng, H, n)
    out, lse = attend(qwm, b, q, first, counts, H, max_count=max(counts))
    gpu_check(b, q, out, lse, first, counts, H)


@pytest.mark.parametrize("batch_size", [500, 513, 1100])
def test_attend_many_prompts(qwm, batch_size):
    """Up to 512 blocks of rows are looked at in one go, more in turn; some are longer than a block and cut."""
    rng = np.random.default_rng(batch_size)
    lengths = [int(rng.integers(17, 80)) for _ in range(batch_size)]
    counts = [int(rng.choice([17, 17, n])) for n in lengths]
    for i in (7, batch_size // 2):
        lengths[i], counts[i] = 900, 600
    b = Batch(qwm, rng, 4, 16, 2, lengths)
    first, n = starts(counts)
    q = rows(rng, 4, n)
    out, lse = attend(qwm, b, q, first, counts, 4, max_count=max(counts))
    gpu_check(b, q, out, lse, first, counts, 4)


@pytest.mark.parametrize("counts", [[1, 3], [1, 150]])
def test_attend_fp32_and_merge(qwm, counts):
    """A sequence attended in two parts, its first pages and the rest, is the sequence attended at once; rows that see
    nothing of a part stay as they were, and rows that see nothing at all are 0 and -inf."""
    rng = np.random.default_rng(5)
    H, kv, page = 4, 2, 32
    lengths = [300, 400]
    b = Batch(qwm, rng, 8, page, kv, lengths)
    first, n = starts(counts)
    q = rows(rng, H, n)
    whole, wl = attend(qwm, b, q, first, counts, H, dtype=torch.float32)
    gpu_check(b, q, whole, wl, first, counts, H, out_eps=2.0 ** -22)
    near, nl = attend(qwm, b, q, first, counts, H, dtype=torch.float32, frames=64)
    far, fl = attend(qwm, b, q, first, counts, H, dtype=torch.float32)
    # the same Queries over the tokens that the window left out, row by row (64-bit weights of the two parts)
    back = torch.exp2(nl.double() - wl.double())
    rest = (whole.double() - near.double() * back[..., None]) / (1 - back)[..., None]
    rl = wl.double() + torch.log2(1 - back)
    out, lse = rest.float().contiguous(), rl.float().contiguous()
    out, lse = attend(qwm, b, q, first, counts, H, out=out, lse=lse, merge=True, frames=64)
    assert float((out - whole).abs().max()) <= 2.0 ** -9 * float(whole.abs().max())
    assert float((lse - wl).abs().max()) <= 2.0 ** -14
    # nothing there yet: merged into (0, -inf) it is the result itself
    out, lse = attend(qwm, b, q, first, counts, H, out=torch.zeros_like(whole), lse=torch.full_like(wl, -math.inf), merge=True)
    assert torch.equal(lse, wl) and float((out - whole).abs().max()) <= 2.0 ** -22 * float(whole.abs().max())
    assert torch.equal(far, whole) and torch.equal(fl, wl)


@pytest.mark.parametrize("count", [2, 100])
def test_attend_growing_logits_and_query_magnitudes(qwm, count):
    """Keys that grow along the sequence raise the running maximum again and again; Queries of any magnitude, and one
    beyond the fp16 range, which is recorded."""
    rng = np.random.default_rng(8)
    b = Batch(qwm, rng, 8, 64, 1, [600], k_scale=6.0)
    q = rows(rng, 1, count, outliers=False)
    for scale in (1.0, 2.0 ** -20, 2.0 ** -100, 0.0):
        x = (q.double() * scale).to(torch.bfloat16)
        out, lse = attend(qwm, b, x, [0], [count], 1)
        assert status(qwm, ctx_of(qwm, 1)) == qwm.QWM_OK
        gpu_check(b, x, out, lse, [0], [count], 1)
    x = q.clone()
    x[0, 1, 5] = 2.0 ** 17
    attend(qwm, b, x, [0], [count], 1)
    assert status(qwm, ctx_of(qwm, 1)) == qwm.QWM_ERR_RANGE


@pytest.mark.parametrize("most", [4, 70])
def test_attend_sequences_left_out(qwm, most):
    """A sequence whose rows begin outside the batch, that has fewer tokens than rows, more rows than was said, or more
    tokens than its pages hold is left out; rows at the batch's end are cut off."""
    rng = np.random.default_rng(2)
    lengths = [100] * 7
    b = Batch(qwm, rng, 8, 16, 2, lengths)
    q = rows(rng, 2, 30)
    want, wl = attend(qwm, b, q, [-1, -1, 4, -1, -1, -1, 28], [0, 0, most // 2, 0, 0, 0, 2], 2, max_count=most)
    b.tab.length[3] = 2
    out, lse = attend(qwm, b, q, [-1, 30, 4, 8, 12, 16, 28], [3, 2, most // 2, 3, 0, -7, most // 2], 2, max_count=most)
    assert status(qwm, ctx_of(qwm, 2)) == qwm.QWM_OK
    # (the last two rows are claimed by sequence 6 and, of 35 rows, by sequence 2)
    assert torch.equal(out[:, :28], want[:, :28]) and torch.equal(lse[:, :28], wl[:, :28])
    for b_, first, counts, err in ((0, 0, most + 1, qwm.QWM_ERR_RANGE), (1, 2, 1, qwm.QWM_ERR_RANGE)):
        f, c = [0] * 7, [0] * 7
        f[b_], c[b_] = first, counts
        if b_ == 1:
            b.tab.length[1] = b.tab.table.shape[1] * 16 + 1
        out, lse = attend(qwm, b, q, f, c, 2, max_count=most)
        assert status(qwm, ctx_of(qwm, 2)) == err
        assert not out.any() and not lse.any()


@pytest.mark.parametrize("counts", [[1, 1], [1, 80]])
def test_attend_page_outside_the_pool_is_recorded(qwm, counts):
    rng = np.random.default_rng(3)
    b = Batch(qwm, rng, 8, 32, 2, [200, 300])
    first, n = starts(counts)
    q = rows(rng, 2, n)
    want, wl = attend(qwm, b, q, first, counts, 2)
    b.tab.table[0, 2] = b.pool.k_codes.shape[0]
    b.tab.table[0, 1] = -1
    out, lse = attend(qwm, b, q, first, counts, 2)
    assert status(qwm, ctx_of(qwm, 2)) == qwm.QWM_ERR_RANGE
    assert torch.equal(out[:, first[1]:], want[:, first[1]:]) and torch.equal(lse[:, first[1]:], wl[:, first[1]:])


def test_attend_layouts_and_workspace(qwm):
    rng = np.random.default_rng(4)
    counts = [40, 1, 3]
    b = Batch(qwm, rng, 4, 64, 2, [500, 90, 128])
    first, n = starts(counts)
    q = rows(rng, 4, n)
    want, wl = attend(qwm, b, q, first, counts, 4)
    for layout in ("head", "padded"):
        x = q.contiguous() if layout == "head" else torch.cat([q, torch.full_like(q[..., :32], 9.0)], -1)[..., :128]
        out = torch.zeros(4, n, 160, dtype=torch.bfloat16, device="cuda")[..., :128]
        out, lse = attend(qwm, b, x, first, counts, 4, out=out)
        assert torch.equal(out, want) and torch.equal(lse, wl)
    need = qwm.qwm_paged_attend_workspace(ctx_of(qwm, 4), b.pool, 40)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = attend(qwm, b, q, first, counts, 4, max_count=40, ws=ws)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    with pytest.raises(qwm.QwmError):
        attend(qwm, b, q, first, counts, 4, max_count=40, ws=ws[:need - 16])


@pytest.mark.parametrize("counts", [[1, 2, 1], [1, 100, 33]])
def test_two_calls_at_once_and_a_replayed_one(qwm, counts):
    """Calls on two streams, each with its workspace, and one replayed from a graph beside them."""
    rng = np.random.default_rng(6)
    b = Batch(qwm, rng, 8, 64, 2, [700, 900, 400])
    first, n = starts(counts)
    qs = [rows(rng, 8, n) for _ in range(3)]
    want = [attend(qwm, b, q, first, counts, 8) for q in qs]
    outs = [torch.zeros(8, n, 128, dtype=torch.bfloat16, device="cuda") for _ in qs]
    lses = [torch.zeros(8, n, dtype=torch.float32, device="cuda") for _ in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    g = torch.cuda.CUDAGraph()
    first, counts = ints(first, torch.int32), ints(counts, torch.int32)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        attend(qwm, b, qs[2], first, counts, 8, out=outs[2], lse=lses[2])
    for _ in range(20):
        for i, s in enumerate(streams):
            attend(qwm, b, qs[i], first, counts, 8, out=outs[i], lse=lses[i], stream=s)
        g.replay()
    torch.cuda.synchronize()
    for (w, wl), o, l in zip(want, outs, lses):
        assert torch.equal(o, w) and torch.equal(l, wl)


# ------------------------------------------------------------------ runs of them together




@pytest.mark.parametrize("norm,rope", [(True, "text"), (True, None), (False, "video"), (False, None)])
@pytest.mark.parametrize("graph", [False, True])
def test_paged_batch(qwm, norm, rope, graph):
    """Sequences that come, grow by prompts, drafts and single tokens, lose drafts and end, through two layers, eager
    or in one captured step replayed; Keys and Values checked through what the pages stand for, outputs against
    64 bits."""
    from bit_kv_cache_qsac_gb300.stream import PagedBatch
    rng = np.random.default_rng(11)
    H, kv, B, rows_, page = 4, 2, 5, 96, 16
    kw = SPECS[rope] if rope else None
    spec = qwm.RopeSpec(**kw) if kw else None
    ctx = ctx_of(qwm, H)
    pb = PagedBatch(ctx, 2, kv, B, 200, 40, rows_, page=page, bits=8, rope=spec, norm=norm)
    wq, wk = (torch.from_numpy(rng.uniform(0.5, 1.5, (128,)).astype(np.float32)).cuda() if norm else None for _ in range(2))
    count, keep = ints([0] * B, torch.int32), ints([2 ** 40] * B)
    q, k, v = ([torch.zeros(h, rows_, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for h in (H, kv, kv))
    outs = [torch.zeros(H, rows_, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lses = [torch.zeros(H, rows_, dtype=torch.float32, device="cuda") for _ in range(2)]

    def step():
        pb.begin(count, keep)
        for i in range(2):
            pb.layer(i, q[i], k[i], v[i], wq, wk, out=outs[i], lse=lses[i])

    step()   # (nothing in it yet)
    if graph:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    ref_pages = paged_ref.Pages(B, -(-200 // page), page, 40)
    stored = [[[] for _ in range(B)] for _ in range(2)]   # per layer and sequence: bf16 (k, v) rows as they came
    plan = [([40, 0, 17, 1, 0], None), ([1, 30, 3, 1, 0], None), ([1, 2, 1, 40, 40], [None, None, 18, None, None]),
            ([1, 1, 0, 60, 1], [30, 0, None, None, None]), ([1, 1, 1, 90, 1], [None] * 5)]
    for counts, keeps in plan:
        count.copy_(ints(counts, torch.int32))
        keeps = [2 ** 40 if x is None else x for x in (keeps or [None] * B)]
        keep.copy_(ints(keeps))
        for i in range(2):
            q[i].copy_(rows(rng, H, rows_))
            k[i].copy_(rows(rng, kv, rows_))
            v[i].copy_(rows(rng, kv, rows_))
        g.replay() if graph else step()
        first, granted, slot, at = ref_pages.update(keeps, counts, rows_)
        assert pb.granted.tolist() == granted and pb.table.length.tolist() == ref_pages.length
        assert pb.check() == qwm.QWM_OK
        for i in range(2):
            for b in range(B):
                old = stored[i][b][:max(0, min(len(stored[i][b]), keeps[b]))]
                new = [(k[i][:, first[b] + t].clone(), v[i][:, first[b] + t].clone()) for t in range(granted[b])]
                stored[i][b] = old + new
                n = ref_pages.length[b]
                assert len(stored[i][b]) == n
                if n == 0:
                    continue
                slots = ints([ref_pages.rows[b][t // page] * page + t % page for t in range(n)])
                hats = [torch.empty(kv, n, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
                qwm.qwm_paged_read(ctx, pb.pools[i], slots, *hats)
                # what is stored is the norm and rotation of what came, within half a step of the 8-bit codes
                for j in range(kv):
                    x = f64(torch.stack([r[0][j] for r in stored[i][b]]))
                    y = paged_ref.norm(x, f64(wk), 1e-6) if norm else x
                    want = turned(y, kw, ref.grid_positions(0, n, *kw.get("grid", (1, 1)))) if kw else y
                    grp = np.repeat(np.abs(want).reshape(n, 4, 32).max(-1), 32, 1)
                    # the step is within 1/8 of the largest over 127; bf16 before and after the codes
                    assert np.all(np.abs(f64(hats[0][j]) - want) <= grp * (1.125 / 127 / 2 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want))
                c = granted[b]
                if not c:
                    continue
                qq = f64(q[i][:, first[b]:first[b] + c])
                if norm:
                    qq = paged_ref.norm(qq, f64(wq), 1e-6)
                if kw:
                    pos = ref.grid_positions(n - c, c, *kw.get("grid", (1, 1)))
                    qq = np.stack([turned(x, kw, pos) for x in qq])
                pool = {t: getattr(pb.pools[i], t).cpu().numpy() for t in ("k_codes", "k_step", "v_codes", "v_step")}
                s = slots.cpu().numpy()
                for h in range(H):
                    take = lambda t: pool[t][s // page, h // 2, s % page]
                    kh, vh = (ref.values(take(x + "_codes"), take(x + "_step"), 8) for x in "kv")
                    want, wl, mag, spread = ref.attend(qq[h], kh, vh, np.arange(n), n - c, 1, ALL, 0, SCALE)
                    # Queries enter in bf16 (2^-8 of their logits' magnitudes), see check() for the rest
                    eps = (2.0 ** -11 + (2.0 ** -8 + 2.0 ** -16) * mag + 2.0 ** -20)[:, None]
                    got = f64(outs[i][h, first[b]:first[b] + c])
                    assert np.all(np.abs(got - want) <= 2 * eps * spread + 2.0 ** -8 * np.abs(want) + 2.0 ** -20)
                    d = np.abs(lses[i][h, first[b]:first[b] + c].double().cpu().numpy() - wl)
                    assert np.all(d <= 2.0 ** -8 * mag + 2.0 ** -16 * mag + 2.0 ** -18)
