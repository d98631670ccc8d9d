"""The paged operators where their arithmetic and their loops are tightest: scales and Queries that underflow,
sequences of up to 2^22 tokens."""
import math

import numpy as np
import pytest

import window_ref as ref
from test_gpu_paged import ALL, SCALE, Batch, ctx_of, ints, rows, starts, status

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


# (bits, kv, count, tokens, tpf, frames, sink): whole items in a share and items cut into parts of several pieces, on
# warp tiles of 8 and of 16 rows and on tiles of 256 and of 512; rows that see nothing of the first or last piece
LONG = [(8, 304, 1, 1 << 22, 1, ALL, 0), (4, 200, 1, (1 << 22) - 100, 1, ALL, 0), (4, 152, 9, 1 << 22, 1, ALL, 0),
        (8, 100, 12, (1 << 22) - 77, 1, 1_500_000, 300), (8, 76, 64, 1 << 22, 1, ALL, 0), (4, 50, 40, (1 << 22) - 1, 1, ALL, 0),
        (4, 76, 300, (1 << 22) - 5, 1, ALL, 0), (8, 50, 600, 3_000_001, 1, 2_900_000, 1000), (8, 76, 300, 3 * (1 << 18) + 150, 1 << 18, 2, 0),
        (4, 304, 20, 2 * (1 << 18) + 7, 1 << 18, 1, 0)]


@pytest.mark.parametrize("mode", ["fp32", "bf16", "merge"])
@pytest.mark.parametrize("case", LONG)
def test_attend_long_sequences(qwm, case, mode):
    """One page of 256 tokens stands in every entry of the table, so that key t is key t % 256 and the definition a
    weighted softmax over 256.  A piece takes 2^18 keys at most: its products are added 16 keys at a time, each off by
    2^-23 of the sum where it is truncated (on warp tiles eight warps take an eighth each), its weights 64 at a time (two
    per lane and 16 keys on warp tiles) by 2^-24; weights are rounded by 2^-11 or 2^-32 of the largest; logits as in
    check() of the other file, in weights and in their sum; 20 pieces and parts joined, 2^-22 each."""
    bits, kv, count, n, tpf, frames, sink = case
    ctx, gen = ctx_of(qwm, kv), torch.Generator(device="cuda").manual_seed(count)
    pool = qwm.PagePool.empty(bits, 256, 1, kv)
    k = torch.randn(kv, 256, 128, device="cuda", generator=gen).to(torch.bfloat16)
    v = (torch.rand(kv, 256, 128, device="cuda", generator=gen) + 0.5).to(torch.bfloat16)
    qwm.qwm_paged_write(ctx, pool, k, v, torch.arange(256, device="cuda"))
    kh, vh = (torch.from_numpy(np.stack([ref.values(getattr(pool, x + "_codes")[0, j].cpu().numpy(), getattr(pool, x + "_step")[0, j].cpu().numpy(), bits)
                                         for j in range(kv)])).cuda() for x in "kv")
    width = -(-n // 256)
    tab = qwm.PageTable(256, torch.zeros(1, width, dtype=torch.int32, device="cuda"), ints([n]), ints([0], torch.int32), ints([0], torch.int32))
    q = torch.randn(kv, count, 128, device="cuda", generator=gen).to(torch.bfloat16)
    out = torch.zeros(kv, count, 128, device="cuda", dtype=torch.bfloat16 if mode == "bf16" else torch.float32)
    lse = torch.zeros(kv, count, device="cuda")
    # how often each row sees each of the 256
    p, j = torch.arange(n - count, n, device="cuda")[:, None], torch.arange(256, device="cuda")
    many = lambda lo, hi: ((hi - 1 - j).div(256, rounding_mode="floor") - (lo - 1 - j).div(256, rounding_mode="floor")).clamp(min=0)
    hi = ((p // tpf + 1) * tpf).clamp(max=n)
    lo = ((p // tpf + 1 - frames) * tpf).clamp(min=sink)
    seen = many(torch.zeros_like(hi), hi.clamp(max=sink)) + many(torch.minimum(lo, hi), hi)
    x = (q.double() @ kh.transpose(1, 2)) * (SCALE * math.log2(math.e)) + torch.log2(seen.double())
    wl = torch.logsumexp(x * math.log(2), -1) / math.log(2)
    w = torch.exp2(x - wl[..., None])
    want, spread = w @ vh, w @ vh.abs()
    mag = (q.double().abs() @ kh.abs().transpose(1, 2)).amax(-1) * SCALE * math.log2(math.e)
    few, piece = count <= 32, 1 << 18
    logits = 2.0 ** -16 * mag + 2.0 ** -20
    sums = piece / 128 * 2.0 ** -24 if few else piece / 64 * 2.0 ** -24
    rel = 2.0 ** -11 + 2 * logits + sums + piece / 16 / (8 if few else 1) * 2.0 ** -23 + 20 * 2.0 ** -22
    far = math.log2(math.e) * sums + logits + 2.0 ** -22 * wl.abs() + 20 * 2.0 ** -22
    bound = rel[..., None] * spread + piece * 2.0 ** -32 * vh.abs().max()
    if mode == "merge":   # into a result of the same weight
        was = torch.randn(kv, count, 128, device="cuda", generator=gen)
        out.copy_(was), lse.copy_(wl)
        want, wl = (want + was.double()) / 2, wl + 1
        bound = bound / 2 + (far[..., None] + 2.0 ** -20) * (spread + was.double().abs())
    qwm.qwm_paged_attend(ctx, pool, tab, q, ints([0], torch.int32), ints([count], torch.int32), SCALE, out, lse=lse, tpf=tpf, frames=frames, sink=sink,
                         max_count=count, merge=mode == "merge")
    assert status(qwm, ctx) == qwm.QWM_OK
    bound = bound + (2.0 ** -8 if mode == "bf16" else 2.0 ** -22) * want.abs()
    assert bool(((out.double() - want).abs() <= bound).all()), float(((out.double() - want).abs() / bound).max())
    assert bool(((lse.double() - wl).abs() <= far + 2.0 ** -22 * wl.abs()).all()), float(((lse.double() - wl).abs() / far).max())


# (bits, lengths, counts, H, kv): whole items and items cut into parts, on warp tiles and on tensor-memory tiles
MERGED = [(8, [40 + 3 * i for i in range(180)], [1 + i % 2 for i in range(180)], 4, 2), (4, [9000, 31], [2, 1], 8, 2), (4, [90 + i for i in range(50)], [40] * 50, 4, 2),
          (8, [6000], [300], 2, 2), (8, [700, 5, 300, 2500], [1, 5, 260, 33], 6, 2)]


@pytest.mark.parametrize("case", MERGED)
def test_attend_merged_into_a_result_over_other_keys(qwm, case):
    """The earlier result is the 64-bit reference's over other keys, rounded to fp32, or made up: nothing seen (-inf,
    with NaN in the output, which is not to be read), far above this call's sums, far below.  The merged mean is off by
    what this call's part is (as check() of the other file) and by what its log-sum-exp shifts between the two: ln 2 of the
    error times the difference."""
    bits, lengths, counts, H, kv = case
    rng, gen = np.random.default_rng(sum(counts)), torch.Generator(device="cuda").manual_seed(sum(counts))
    b = Batch(qwm, rng, bits, 16, kv, lengths)
    first, n = starts(counts, gap=1)
    q = rows(rng, H, n)
    far_k, far_v = (torch.randn(H, 77, 128, device="cuda", generator=gen).double() for _ in range(2))
    x = q.double() @ far_k.transpose(1, 2) * (SCALE * math.log2(math.e))
    lse = (torch.logsumexp(x * math.log(2), -1) / math.log(2)).float()
    out = (torch.softmax(x * math.log(2), -1) @ far_v).float()
    kind = torch.arange(n, device="cuda")[None] * 3 + torch.arange(H, device="cuda")[:, None]
    lse[kind % 5 == 1], out[kind % 5 == 1] = -math.inf, math.nan
    lse[kind % 5 == 2] += 60.0
    lse[kind % 5 == 3] -= 60.0
    was, wasl = out.clone(), lse.clone()
    ctx = ctx_of(qwm, H)
    for most in (max(counts), None):
        out.copy_(was), lse.copy_(wasl)
        qwm.qwm_paged_attend(ctx, b.pool, b.tab, q, ints(first, torch.int32), ints(counts, torch.int32), SCALE, out, lse=lse, merge=True, max_count=most)
        assert status(qwm, ctx) == qwm.QWM_OK
        mine = torch.zeros(n, dtype=torch.bool, device="cuda")
        for i, (c, m) in enumerate(zip(counts, lengths)):
            f = slice(first[i], first[i] + c)
            mine[f] = True
            k, v = (torch.from_numpy(y[i]).cuda().repeat_interleave(H // kv, 0) for y in (b.k, b.v))
            see = torch.arange(m, device="cuda") <= torch.arange(m - c, m, device="cuda")[:, None]
            x = (q[:, f].double() @ k.transpose(1, 2) * (SCALE * math.log2(math.e))).masked_fill(~see, -math.inf)
            wl = torch.logsumexp(x * math.log(2), -1) / math.log(2)
            w = torch.exp2(x - wl[..., None])
            part, spread = w @ v, w @ v.abs()
            mag = (q[:, f].double().abs() @ k.abs().transpose(1, 2)).amax(-1) * SCALE * math.log2(math.e)
            bound = 2 * (2.0 ** -11 + 2.0 ** -16 * mag + 2.0 ** -20)[..., None] * spread + m * 2.0 ** -31 * v.abs().max()
            d = 2.0 ** -16 * mag + 2.0 ** -20 + 2.0 ** -22 * wl.abs()
            lp, prev = wasl[:, f].double(), was[:, f].double().nan_to_num(0.0)
            want_l = torch.logaddexp2(lp, wl)
            up, ut = torch.exp2(lp - want_l)[..., None], torch.exp2(wl - want_l)[..., None]
            want = up * prev + ut * part
            err = ut * bound + math.log(2) * (d + 2.0 ** -22 * lp.abs().nan_to_num(0, 0, 0))[..., None] * up * ut * (prev - part).abs() + 2.0 ** -20 * (up * prev.abs() + ut * part.abs())
            assert bool(((out[:, f].double() - want).abs() <= err + 2.0 ** -30).all()), i
            assert bool(((lse[:, f].double() - want_l).abs() <= d + 2.0 ** -22 * want_l.abs() + 2.0 ** -20).all()), i
        assert torch.equal(out[:, ~mine].view(torch.int32), was[:, ~mine].view(torch.int32)) and torch.equal(lse[:, ~mine], wasl[:, ~mine])


# ------------------------------------------------------------------ offsets beyond 32 bits


@pytest.mark.parametrize("bits,counts", [(8, [1, 3]), (8, [40, 300]), (4, [5, 2]), (4, [1, 130])])
def test_pools_beyond_four_gigabytes(qwm, bits, counts):
    """Pages on both sides of 2^32 bytes of codes (and 2^31 of rows' channels): written, read back and attended they are
    what the same tokens are in a small pool."""
    rng, kv, H, page, lengths = np.random.default_rng(bits), 8, 16, 64, [700, 900]
    pages = 70_000 if bits == 8 else 140_000   # 4.6 GB of codes each
    need = sum(-(-n // page) for n in lengths)
    large, small = qwm.PagePool.empty(bits, page, pages, kv), qwm.PagePool.empty(bits, page, need, kv)
    where = torch.from_numpy(np.concatenate([rng.permutation(need)[:need // 2], pages - 1 - rng.permutation(need)[:need - need // 2]])).cuda()
    where = where[torch.from_numpy(rng.permutation(need)).cuda()]
    n = sum(lengths)
    k, v = rows(rng, kv, n), rows(rng, kv, n)
    at = torch.cat([torch.arange(m) + off * page for m, off in ((lengths[0], 0), (lengths[1], -(-lengths[0] // page)))]).cuda()
    first_pages = [-(-m // page) for m in lengths]
    tabs, ctx = [], ctx_of(qwm, H)
    hats = []
    for pool, order in ((large, where), (small, torch.arange(need, device="cuda"))):
        slot = order[at // page] * page + at % page
        qwm.qwm_paged_write(ctx, pool, k, v, slot)
        hats.append([torch.empty(kv, n, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)])
        qwm.qwm_paged_read(ctx, pool, slot, *hats[-1])
        t = torch.full((2, max(first_pages)), -1, dtype=torch.int32, device="cuda")
        t[0, :first_pages[0]], t[1, :first_pages[1]] = order[:first_pages[0]].int(), order[first_pages[0]:].int()
        tabs.append(qwm.PageTable(page, t, ints(lengths), torch.zeros(pool.k_codes.shape[0], dtype=torch.int32, device="cuda"), ints([0], torch.int32)))
    assert int(where.max()) * kv * page * 128 * bits // 8 > 2 ** 32
    assert all(torch.equal(a, b) and bool(a.any()) for a, b in zip(*hats))
    first, m = starts(counts)
    q, got = rows(rng, H, m), []
    for pool, tab in ((large, tabs[0]), (small, tabs[1])):
        out, lse = torch.zeros(H, m, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(H, m, device="cuda")
        qwm.qwm_paged_attend(ctx, pool, tab, q, ints(first, torch.int32), ints(counts, torch.int32), SCALE, out, lse=lse, max_count=max(counts))
        got.append((out, lse))
    assert status(qwm, ctx) == qwm.QWM_OK
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and bool(got[0][0].any())


@pytest.mark.parametrize("head_major", [False, True])
def test_packed_batches_beyond_32_bits(qwm, head_major):
    """The last rows of a batch whose activations pass 2^31 elements (and 2^32 bytes): normed, turned, stored and attended they
    are what the same rows are in a small batch."""
    rng, H, n, counts, lengths = np.random.default_rng(3), 40, 440_000, [2, 60], [300, 400]
    ctx, spec, live = ctx_of(qwm, H), qwm.RopeSpec((128, 0, 0), theta=1e6, pairing="half"), sum(counts)
    lot = lambda dtype=torch.bfloat16: (torch.zeros(H, n, 128, dtype=dtype, device="cuda") if head_major
                                        else torch.zeros(n, H, 128, dtype=dtype, device="cuda").permute(1, 0, 2))
    x, ready, out = lot(), lot(), lot()
    some = rows(rng, H, live)
    x[:, -live:] = some
    at = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    at[-live:] = torch.arange(live, device="cuda") + 7
    w = torch.from_numpy(rng.uniform(0.5, 1.5, (H, 128)).astype(np.float32)).cuda()
    qwm.qwm_norm_rope(ctx, spec, x[None], w, 1e-6, ready[None], at=at[None])
    want = torch.empty(1, H, live, 128, dtype=torch.bfloat16, device="cuda")
    qwm.qwm_norm_rope(ctx, spec, some[None], w, 1e-6, want, at=at[None, -live:].contiguous())
    assert torch.equal(ready[:, -live:], want[0]) and not ready[:, :-live].any()
    b = Batch(qwm, rng, 8, 32, H, lengths)
    pools = [qwm.PagePool.empty(8, 32, 4, H) for _ in range(2)]
    slot = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    slot[-live:] = torch.arange(live, device="cuda") * 2
    qwm.qwm_paged_write(ctx, pools[0], x, x, slot, at=at, rope=spec, weight=w)
    qwm.qwm_paged_write(ctx, pools[1], some, some, slot[-live:].contiguous(), at=at[-live:].contiguous(), rope=spec, weight=w)
    assert all(torch.equal(getattr(pools[0], t), getattr(pools[1], t)) for t in ("k_codes", "k_step", "v_codes", "v_step")) and pools[0].k_codes.any()
    small, lse = torch.zeros(H, live, 128, dtype=torch.bfloat16, device="cuda"), [torch.zeros(H, m, device="cuda") for m in (n, live)]
    qwm.qwm_paged_attend(ctx, b.pool, b.tab, ready, ints([n - live, n - live + counts[0]], torch.int32), ints(counts, torch.int32), SCALE, out, lse=lse[0],
                         max_count=max(counts))
    qwm.qwm_paged_attend(ctx, b.pool, b.tab, want[0], ints([0, counts[0]], torch.int32), ints(counts, torch.int32), SCALE, small, lse=lse[1], max_count=max(counts))
    assert status(qwm, ctx) == qwm.QWM_OK
    assert torch.equal(out[:, -live:], small) and torch.equal(lse[0][:, -live:], lse[1]) and bool(small.any())
    assert not out[:, :-live].any() and not lse[0][:, :-live].any()
