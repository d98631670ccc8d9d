"""Host-side checks of the paged cache (no GPU): every refusal, which comes before the first CUDA call, and
the reference's own properties."""
import ctypes as C

import numpy as np
import pytest

import paged_ref


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


OK = 0x7f00000000   # a stand-in pointer: 16-byte aligned, never read


def _tab(qwm, **kw):
    d = dict(page=64, batch=3, width=10, pages=40, table=OK, length=OK, free_list=OK, free_count=OK)
    d.update(kw)
    return qwm.qwm_page_table(**d)


def _pool(qwm, **kw):
    d = dict(bits=8, page=64, pages=40, kv_heads=4, k_codes=OK, v_codes=OK, k_step=OK, v_step=OK)
    d.update(kw)
    return qwm.qwm_page_pool(**d)


def _st(qwm, batch=0, head=128, token=128 * 8):
    return qwm.qwm_strides(batch, head, token)


BAD_TABLES = [(dict(page=8), "QWM_ERR_UNSUPPORTED"), (dict(page=48), "QWM_ERR_UNSUPPORTED"), (dict(page=512), "QWM_ERR_UNSUPPORTED"),
              (dict(batch=0), "QWM_ERR_ARG"), (dict(batch=4097), "QWM_ERR_SHAPE"), (dict(width=0), "QWM_ERR_ARG"),
              (dict(width=(1 << 16) + 1), "QWM_ERR_SHAPE"), (dict(table=None), "QWM_ERR_ARG"), (dict(length=None), "QWM_ERR_ARG"),
              (dict(table=OK + 2), "QWM_ERR_ALIGN"), (dict(length=OK + 4), "QWM_ERR_ALIGN")]
BAD_STACKS = [(dict(pages=0), "QWM_ERR_ARG"), (dict(free_list=None), "QWM_ERR_ARG"), (dict(free_count=None), "QWM_ERR_ARG"),
              (dict(free_list=OK + 2), "QWM_ERR_ALIGN"), (dict(free_count=OK + 1), "QWM_ERR_ALIGN")]
BAD_POOLS = [(dict(bits=2), "QWM_ERR_UNSUPPORTED"), (dict(bits=16), "QWM_ERR_UNSUPPORTED"), (dict(page=24), "QWM_ERR_UNSUPPORTED"),
             (dict(pages=0), "QWM_ERR_ARG"), (dict(kv_heads=0), "QWM_ERR_ARG"), (dict(kv_heads=-2), "QWM_ERR_ARG"),
             (dict(k_codes=None), "QWM_ERR_ARG"), (dict(v_step=None), "QWM_ERR_ARG"), (dict(v_codes=OK + 8), "QWM_ERR_ALIGN"),
             (dict(k_step=OK + 4), "QWM_ERR_ALIGN")]


def _attend(qwm, ctx=None, pool=None, tab=None, q=OK, qs=None, n=5, first=OK, count=OK, most=5, tpf=1, frames=8, sink=0, scale=1.0, out=OK,
            os=None, f32=0, lse=None, merge=0, ws=OK, nws=1 << 40, **kw):
    return qwm.raw_library().qwm_paged_attend(kw.get("context", ctx or _ctx(qwm)), pool or _pool(qwm), tab or _tab(qwm), q, qs or _st(qwm), n, first,
                                              count, most, tpf, frames, sink, scale, out, os or _st(qwm), f32, lse, merge, ws, nws, None)


@pytest.mark.parametrize("kw,err", BAD_TABLES)
def test_table_refusals(qwm, kw, err):
    lib, ctx, t, want = qwm.raw_library(), _ctx(qwm), _tab(qwm, **kw), getattr(qwm, err)
    assert lib.qwm_pages_reset(ctx, t, None) == want
    assert lib.qwm_pages_update(ctx, t, OK, OK, 3, OK, OK, OK, OK, None) == want
    assert _attend(qwm, tab=t) == want


@pytest.mark.parametrize("kw,err", BAD_STACKS)
def test_stack_refusals(qwm, kw, err):
    lib, ctx, t, want = qwm.raw_library(), _ctx(qwm), _tab(qwm, **kw), getattr(qwm, err)
    assert lib.qwm_pages_reset(ctx, t, None) == want
    assert lib.qwm_pages_update(ctx, t, OK, OK, 3, OK, OK, OK, OK, None) == want


@pytest.mark.parametrize("kw,err", BAD_POOLS)
def test_pool_refusals(qwm, kw, err):
    lib, ctx, p, s, want = qwm.raw_library(), _ctx(qwm), _pool(qwm, **kw), _st(qwm), getattr(qwm, err)
    assert lib.qwm_paged_write(ctx, p, OK, s, OK, s, 3, OK, None, None, None, 0, None, 0, 0.0, None) == want
    assert lib.qwm_paged_read(ctx, p, OK, 3, OK, OK, None) == want
    assert _attend(qwm, pool=p) == want


def test_update_refusals(qwm):
    lib, t = qwm.raw_library(), _tab(qwm)

    def call(ctx=_ctx(qwm), keep=OK, count=OK, n=3, first=OK, granted=OK, slot=OK, at=OK):
        return lib.qwm_pages_update(ctx, t, keep, count, n, first, granted, slot, at, None)
    assert call(keep=None, count=None, n=0) == qwm.QWM_OK
    for kw in (dict(ctx=None), dict(n=-1), dict(first=None), dict(granted=None), dict(slot=None), dict(at=None), dict(count=None)):
        assert call(**kw) == qwm.QWM_ERR_ARG, kw
    for kw in (dict(keep=OK + 4), dict(count=OK + 2), dict(first=OK + 1), dict(granted=OK + 2), dict(slot=OK + 4), dict(at=OK + 4)):
        assert call(**kw) == qwm.QWM_ERR_ALIGN, kw
    assert call(n=(1 << 24) + 1) == qwm.QWM_ERR_SHAPE
    assert lib.qwm_pages_reset(None, t, None) == qwm.QWM_ERR_ARG
    assert lib.qwm_pages_update(_ctx(qwm), None, OK, OK, 3, OK, OK, OK, OK, None) == qwm.QWM_ERR_ARG


def test_write_refusals(qwm):
    lib, p, s = qwm.raw_library(), _pool(qwm), _st(qwm)
    r = qwm.RopeSpec((16, 0, 0))

    def call(ctx=_ctx(qwm), k=OK, ks=s, v=OK, vs=s, n=3, slot=OK, rope=None, at=None, pos=None, norm=0, weight=None, per_head=0, eps=0.0):
        return lib.qwm_paged_write(ctx, p, k, ks, v, vs, n, slot, rope, at, pos, norm, weight, per_head, eps, None)
    assert call(n=0) == qwm.QWM_OK
    for kw in (dict(ctx=None), dict(n=-1), dict(k=None), dict(v=None), dict(slot=None), dict(at=OK), dict(pos=OK), dict(rope=r), dict(norm=2),
               dict(weight=OK), dict(norm=1, eps=-1.0), dict(norm=1, eps=float("nan")), dict(norm=1, eps=float("inf")), dict(norm=1, per_head=2),
               dict(ks=_st(qwm, head=-8)), dict(vs=None)):
        assert call(**kw) == qwm.QWM_ERR_ARG, kw
    for kw in (dict(k=OK + 2), dict(vs=_st(qwm, token=130)), dict(slot=OK + 4), dict(rope=r, at=OK + 4), dict(rope=r, at=OK, pos=OK + 2),
               dict(norm=1, weight=OK + 4)):
        assert call(**kw) == qwm.QWM_ERR_ALIGN, kw
    assert call(n=(1 << 24) + 1) == qwm.QWM_ERR_SHAPE
    bad = qwm.RopeSpec((16, 0, 0))
    bad.rot = 130
    assert call(rope=bad, at=OK) == qwm.QWM_ERR_SHAPE


def test_read_refusals(qwm):
    lib, ctx, p = qwm.raw_library(), _ctx(qwm), _pool(qwm)
    assert lib.qwm_paged_read(ctx, p, OK, 0, OK, OK, None) == qwm.QWM_OK
    assert lib.qwm_paged_read(ctx, p, OK, 3, None, None, None) == qwm.QWM_OK
    for a in ((None, p, OK, 3, OK, OK), (ctx, None, OK, 3, OK, OK), (ctx, p, None, 3, OK, OK), (ctx, p, OK, -1, OK, OK)):
        assert lib.qwm_paged_read(*a, None) == qwm.QWM_ERR_ARG
    for a in ((ctx, p, OK + 4, 3, OK, OK), (ctx, p, OK, 3, OK + 8, OK), (ctx, p, OK, 3, OK, OK + 2)):
        assert lib.qwm_paged_read(*a, None) == qwm.QWM_ERR_ALIGN
    assert lib.qwm_paged_read(ctx, p, OK, (1 << 24) + 1, OK, OK, None) == qwm.QWM_ERR_SHAPE


def test_norm_rope_refusals(qwm):
    lib, s, r = qwm.raw_library(), _st(qwm, batch=1 << 14), qwm.RopeSpec((16, 0, 0))

    def call(ctx=_ctx(qwm), r=r, x=OK, xs=s, b=2, h=8, n=3, start=OK, at=None, pos=None, weight=OK, per_head=0, eps=1e-6, out=OK + 4096, os=s):
        return lib.qwm_norm_rope(ctx, r, x, xs, b, h, n, start, at, pos, weight, per_head, eps, out, os, None)
    for kw in (dict(n=0), dict(b=0), dict(h=0)):
        assert call(**kw) == qwm.QWM_OK, kw
    for kw in (dict(ctx=None), dict(x=None), dict(out=None), dict(start=None), dict(at=OK), dict(n=-1), dict(b=-1), dict(r=None, pos=OK),
               dict(out=OK, os=_st(qwm, batch=1 << 20)), dict(os=_st(qwm, token=128)), dict(xs=None), dict(per_head=-1), dict(eps=-0.5),
               dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(**kw) == qwm.QWM_ERR_ARG, kw
    for kw in (dict(x=OK + 2), dict(xs=_st(qwm, token=4)), dict(pos=OK + 1), dict(weight=OK + 4), dict(start=OK + 4), dict(start=None, at=OK + 2)):
        assert call(**kw) == qwm.QWM_ERR_ALIGN, kw
    for kw in (dict(n=(1 << 24) + 1), dict(b=1 << 17), dict(b=60000, n=1 << 20)):
        assert call(**kw) == qwm.QWM_ERR_SHAPE, kw


def test_attend_refusals(qwm):
    assert _attend(qwm, n=0) == qwm.QWM_OK and _attend(qwm, most=0) == qwm.QWM_OK
    for kw in (dict(context=None), dict(n=-1), dict(most=-1), dict(q=None), dict(out=None), dict(first=None), dict(count=None), dict(tpf=0),
               dict(frames=0), dict(sink=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(f32=2),
               dict(merge=2), dict(merge=1), dict(merge=1, f32=1), dict(merge=1, lse=OK), dict(os=_st(qwm, token=0)), dict(os=_st(qwm, head=120)),
               dict(tab=_tab(qwm, page=32)), dict(ws=None)):
        assert _attend(qwm, **kw) == qwm.QWM_ERR_ARG, kw
    for kw in (dict(q=OK + 8), dict(out=OK + 4), dict(qs=_st(qwm, head=4)), dict(lse=OK + 2), dict(first=OK + 2), dict(count=OK + 1)):
        assert _attend(qwm, **kw) == qwm.QWM_ERR_ALIGN, kw
    assert _attend(qwm, ws=OK + 8) in (qwm.QWM_ERR_ARG, qwm.QWM_ERR_ALIGN)
    for kw in (dict(pool=_pool(qwm, kv_heads=3)), dict(n=(1 << 24) + 1), dict(most=(1 << 24) + 1), dict(frames=(1 << 31) + 1), dict(tpf=(1 << 31) + 1)):
        assert _attend(qwm, **kw) == qwm.QWM_ERR_SHAPE, kw
    lib = qwm.raw_library()
    assert lib.qwm_paged_attend_workspace(_ctx(qwm), _pool(qwm, kv_heads=3), 5) == 0
    assert lib.qwm_paged_attend_workspace(_ctx(qwm), _pool(qwm), 0) == 0
    assert lib.qwm_paged_attend_workspace(None, _pool(qwm), 5) == 0


def test_binding_refuses_host_tensors_and_shapes(qwm):
    import torch

    class Ctx:
        handle, heads, device = None, 8, torch.device("cuda", 0)
    x = torch.zeros(1, 8, 3, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        qwm.qwm_norm_rope(Ctx, None, x, None, 1e-6, x)
    pool = qwm.PagePool.empty(8, 16, 2, 8, device="cpu")
    with pytest.raises(TypeError):
        qwm.qwm_paged_write(Ctx, pool, x[0], x[0], torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        qwm.qwm_pages_update(Ctx, qwm.PageTable.empty(1, 1, 16, 2, device="cpu"), keep=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError):
        qwm.PagePool.empty(2, 16, 2, 8, device="cpu")


def test_reference_pages_are_kept_apart():
    """The reference's own properties: no page is in two places, and every page is somewhere."""
    rng = np.random.default_rng(4)
    ref = paged_ref.Pages(7, 5, 16, 20)
    for _ in range(50):
        keep = [int(rng.integers(0, 80)) for _ in range(7)]
        count = [int(rng.integers(-2, 40)) for _ in range(7)]
        first, granted, slot, at = ref.update(keep, count, int(rng.integers(0, 200)))
        held = [p for r in ref.rows for p in r] + ref.free
        assert sorted(held) == list(range(20))
        assert all(len(r) == -(-n // 16) <= 5 for r, n in zip(ref.rows, ref.length))
        live = [s for s in slot if s >= 0]
        assert len(live) == len(set(live)) == sum(granted)


def test_attend_refuses_more_rows_than_items_can_number(qwm):
    many, pool = _ctx(qwm, heads=1 << 17), _pool(qwm, kv_heads=1 << 15)
    wide = _st(qwm, token=128 << 17)
    assert _attend(qwm, ctx=many, pool=pool, qs=wide, os=wide, n=(1 << 19) + 1) == qwm.QWM_ERR_SHAPE
    assert _attend(qwm, ctx=many, pool=pool, qs=wide, os=wide, n=1 << 19, ws=None) == qwm.QWM_ERR_ARG   # (the next check's)
