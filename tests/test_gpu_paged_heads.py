"""The loops of the norm, write and read-back kernels over the heads of a block: calls large enough for several heads
a block (all smaller ones give each head a block of its own), odd numbers of heads, more than 64, weights per head,
and rows whose squares leave fp32's range among the others."""
import math

import numpy as np
import pytest

import paged_ref
import window_ref as ref
from test_gpu_paged import SPECS, ctx_of, f64, ints, norm_bound, rows, status, turned

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qwm():
    import bit_kv_cache_qsac_gb300 as q
    return q


def heads_a_block(tiles, heads, per_sm, most):
    """As the launches choose them."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    parts = max(1, min(heads, (sms * per_sm + tiles // 2) // tiles))
    return min(most, -(-heads // parts))


def heads_of_norm(heads, n):
    return heads_a_block(-(-n // 16), heads, 12, 64)


def heads_of_write(heads, n, rope):
    return heads_a_block(-(-n // 16), heads, 9 if rope else 20, 64)


def heads_of_read(heads, n):
    return heads_a_block(-(-n // 32), heads, 40, heads)


def weights(rng, kind, h):
    return torch.from_numpy(rng.uniform(0.2, 2.0, (h, 128) if kind == "heads" else (128,)).astype(np.float32)).cuda() if kind else None


def many_rows(seed, h, n):
    """bf16 rows [h][n][128] as a projection leaves them (token-major)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, h, 128, generator=gen, device="cuda").to(torch.bfloat16).permute(1, 0, 2)


ODD = [2.0 ** 100, 2.0 ** 125, 2.0 ** -60, 2.0 ** -70, 2.0 ** -100, 2.0 ** -125, 0.0, math.inf, math.nan]


def with_odd_rows(x):
    """Rows of magnitudes whose squares overflow or vanish, of zeros, and rows with an infinity or a NaN, a different
    one in each head and token, two neighbouring heads of a token among them; returns the changed tokens of each head."""
    h, n = x.shape[:2]
    where = {}
    for i in range(min(h, 3 * len(ODD))):
        head, token = i * h // min(h, 3 * len(ODD)), (7919 * (i // 2) + 13) % n
        f = ODD[i % len(ODD)]
        if math.isfinite(f):
            x[head, token] = (x[head, token].double() * f).clamp(-2.0 ** 127, 2.0 ** 127).to(torch.bfloat16)
        else:
            x[head, token, (29 * i) % 128] = f
        where.setdefault(head, []).append(token)
    return where


# ------------------------------------------------------------------ norm and rotation


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("name", ["video", "text", "partial", "none"])
@pytest.mark.parametrize("h,n,kind,inplace", [(40, 10800, "heads", False), (41, 10801, "heads", True), (40, 10799, "one", True), (9, 30000, None, False),
                                              (130, 40000, "heads", False), (3, 20005, "heads", True)])
def test_norm_rope_several_heads_a_block(qwm, name, h, n, kind, inplace, odd):
    """Every row is, bit for bit, that of its head alone (a block of its own), and sampled rows of every head are those
    of the 64-bit reference."""
    assert heads_of_norm(h, n) > 1 and heads_of_norm(1, n) == 1
    kw, rng = SPECS[name], np.random.default_rng(h + n)
    x, w, spec = many_rows(h, h, n), weights(rng, kind, h), qwm.RopeSpec(**kw) if kw else None
    where = with_odd_rows(x) if odd else {}
    was, ctx, start = x.clone(), ctx_of(qwm, 1), ints([70_001]) if kw else None
    out = x if inplace else torch.full((n, h, 128), 7.0, dtype=torch.bfloat16, device="cuda").permute(1, 0, 2)
    qwm.qwm_norm_rope(ctx, spec, x[None], w, 1e-6, out[None], start=start)
    alone = torch.empty(1, 1, n, 128, dtype=torch.bfloat16, device="cuda")
    for j in range(h):
        qwm.qwm_norm_rope(ctx, spec, was[None, j:j + 1], w[j].contiguous() if kind == "heads" else w, 1e-6, alone, start=start)
        assert torch.equal(out[j].view(torch.int16), alone[0, 0].view(torch.int16)), j
    grid = (kw or {}).get("grid", (1, 1))
    for j in range(h):
        take = sorted(set(rng.integers(0, n, 6).tolist() + where.get(j, [])))
        y = paged_ref.norm(f64(was[j, take]), f64(w[j] if kind == "heads" else w) if kind else 1.0, float(np.float32(1e-6)))
        infinite = np.isinf(f64(was[j, take]))
        y[infinite.any(-1)] = 0.0   # finite over infinite, and
        y[infinite] = np.nan        # infinite over infinite
        pos = np.concatenate([ref.grid_positions(70_001 + t, 1, *grid) for t in take])
        want = turned(y, kw, pos) if kw else y
        got, nan = f64(out[j, take]), np.isnan(want)
        assert np.array_equal(nan, np.isnan(got)), j
        # results below the normal numbers keep fp32's grid of 2^-149, 2^-133 in bf16
        assert np.all((np.abs(got - want) <= norm_bound(y, want, kw) + 2.0 ** -133)[~nan]), j


# ------------------------------------------------------------------ the paged cache


def slots(rng, n, page, pages, skip):
    """Distinct slots of scattered pages, some rows skipped."""
    order, i = rng.permutation(pages), np.arange(n)
    s = order[i // page] * page + i % page
    s[i % 97 == 5] = -1 if skip else s[i % 97 == 5]
    return torch.from_numpy(s.astype(np.int64)).cuda()


def images(pool):
    return [getattr(pool, t) for t in ("k_codes", "k_step", "v_codes", "v_step")]


def stand_for(x, bits):
    """Codes and steps of rows [n][128]: what leaves the range is cut, a NaN becomes 0."""
    top = ref.Q[bits] * ref.STEP_TOP[bits]
    q, step = ref.quantise(np.where(np.isnan(x), 0.0, np.clip(x, -top, top)), bits)
    return ref.pack(q, bits), step


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("name,kind,h,n,page", [("video", "heads", 40, 10800, 128), ("text", "one", 8, 30011, 64), ("text", "heads", 41, 5001, 16),
                                                (None, "heads", 40, 8001, 256), (None, None, 8, 60000, 64), ("partial", None, 13, 20000, 32),
                                                ("text", "heads", 130, 40000, 64)])
def test_write_and_read_several_heads_a_block(qwm, name, kind, h, n, page, bits):
    """The pages are, byte for byte, those of the same rows written in pieces that give each head a block of its own;
    sampled rows of every head are the quantised rows of the norm and rotation alone; read back, they are what the
    same pieces give, and the reference's values."""
    rope = name is not None
    assert heads_of_write(h, n, rope) > 1 and heads_of_read(h, n) > 1
    kw, rng = SPECS[name] if rope else None, np.random.default_rng(n + bits)
    spec, w, ctx = qwm.RopeSpec(**kw) if rope else None, weights(rng, kind, h), ctx_of(qwm, 1)
    k, v = many_rows(1, h, n), many_rows(2, h, n)
    pages = -(-n // page) + 2
    slot = slots(rng, n, page, pages, True)
    at = torch.arange(n, device="cuda") * 3 + 1000 if rope else None
    pool, again = (qwm.PagePool.empty(bits, page, pages, h) for _ in range(2))
    for t in images(pool) + images(again):
        t.fill_(0x33)
    qwm.qwm_paged_write(ctx, pool, k, v, slot, at=at, rope=spec, weight=w, eps=1e-6)
    piece = 512 if h < 100 else 128
    assert heads_of_write(h, piece, rope) == heads_of_read(h, piece) == 1
    for i in range(0, n, piece):
        cut = slice(i, min(n, i + piece))
        qwm.qwm_paged_write(ctx, again, k[:, cut], v[:, cut], slot[cut], at=at[cut].contiguous() if rope else None, rope=spec, weight=w, eps=1e-6)
    assert status(qwm, ctx) == qwm.QWM_OK
    for a, b in zip(images(pool), images(again)):
        assert torch.equal(a, b)
    hats = [torch.full((h, n, 128), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    qwm.qwm_paged_read(ctx, pool, slot, *hats)
    for i in range(0, n, piece):
        cut = slice(i, min(n, i + piece))
        some = [torch.empty(h, cut.stop - i, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        qwm.qwm_paged_read(ctx, pool, slot[cut], *some)
        assert all(torch.equal(a[:, cut], b) for a, b in zip(hats, some))
    ready = k.clone()
    if kind:
        qwm.qwm_norm_rope(ctx, spec, k[None], w, 1e-6, ready[None], at=at[None] if rope else None)
    elif rope:
        pos = torch.stack([at // math.prod(kw["grid"]), at // kw["grid"][1] % kw["grid"][0], at % kw["grid"][1]], -1).to(torch.int32)
        qwm.qwm_rope(ctx, spec, k[None], ints([0]), ready[None], pos=pos[None])
    take = torch.from_numpy(np.unique(np.append(rng.integers(0, n, 9), [5, n - 1]))).cuda()
    s = slot[take].tolist()
    for x, (codes, step), hat in ((ready, images(pool)[:2], hats[0]), (v, images(pool)[2:], hats[1])):
        for j in range(h):
            c, st = stand_for(f64(x[j, take]), bits)
            val = ref.bf16(ref.values(c, st, bits))
            for i, where in enumerate(s):
                got = f64(hat[j, take[i]])
                if where < 0:
                    assert not got.any()
                    continue
                p = (where // page, j, where % page)
                assert np.array_equal(codes[p].cpu().numpy(), c[i]) and np.array_equal(step[p].cpu().numpy(), st[i]), (j, i)
                assert np.array_equal(got, val[i])
    held = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
    held[slot[slot >= 0]] = True
    for t in images(pool):
        assert bool((t.transpose(1, 2).flatten(0, 1)[~held] == 0x33).all())


@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("name,kind,h,n", [("video", "heads", 40, 5001), ("text", None, 40, 700), ("text", "one", 3, 40), (None, "heads", 41, 3001), (None, None, 2, 33),
                                           ("partial", "heads", 130, 4000)])
def test_write_rows_beyond_the_range_of_squares(qwm, name, kind, h, n, bits, eps):
    """Keys whose squares leave fp32's range, zeros, infinities and NaN beside ordinary rows and skipped ones, several
    heads a block and one: the codes are those of qwm_norm_rope's output, Values and other slots as without them, and what
    is no number is recorded."""
    rope = name is not None
    kw, rng = SPECS[name] if rope else None, np.random.default_rng(n)
    spec, w, ctx, page = qwm.RopeSpec(**kw) if rope else None, weights(rng, kind, h), ctx_of(qwm, 1), 32
    k, v = many_rows(3, h, n), many_rows(4, h, n)
    where = with_odd_rows(k)
    if not rope and n == 33:   # whole warps of such rows, one of them skipped
        k[1, :20] = (k[1, :20].double() * 2.0 ** 110).to(torch.bfloat16)
        where[1] = where.get(1, []) + list(range(20))
    pages = -(-n // page) + 1
    slot = slots(rng, n, page, pages, True)
    pos = torch.from_numpy(rng.integers(0, 1000, (n, 3)).astype(np.int32)).cuda() if name == "partial" else None
    at = torch.arange(n, device="cuda") + 50 if rope else None
    pool = qwm.PagePool.empty(bits, page, pages, h)
    for t in images(pool):
        t.fill_(0x33)
    qwm.qwm_paged_write(ctx, pool, k, v, slot, at=at, rope=spec, pos=pos, norm=True, weight=w, eps=eps)
    ready = torch.empty(1, h, n, 128, dtype=torch.bfloat16, device="cuda")
    recorded = status(qwm, ctx)
    qwm.qwm_norm_rope(ctx, spec, k[None], w, eps, ready, at=at[None] if rope else None, pos=pos[None] if pos is not None else None)
    s = slot.tolist()
    bad = bool((ready[0, :, slot >= 0].isnan()).any())
    assert recorded == (qwm.QWM_ERR_RANGE if bad else qwm.QWM_OK)
    c = [t.cpu().numpy() for t in images(pool)]
    for j in range(h):
        near = {min(n - 1, max(0, t + d)) for t in where.get(j, []) for d in (-16, -1, 0, 1, 16)}
        take = sorted(near | set(rng.integers(0, n, 4).tolist()))
        for x, codes, step in ((ready[0, j], c[0], c[1]), (v[j], c[2], c[3])):
            want, st = stand_for(f64(x[take]), bits)
            for i, t in enumerate(take):
                if s[t] >= 0:
                    p = (s[t] // page, j, s[t] % page)
                    assert np.array_equal(codes[p], want[i]) and np.array_equal(step[p], st[i]), (j, t)
    held = np.zeros(pages * page, bool)
    held[[x for x in s if x >= 0]] = True
    for t in c:
        assert np.all(np.swapaxes(t, 1, 2).reshape(pages * page, h, -1)[~held] == 0x33)
