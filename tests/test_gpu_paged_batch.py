"""PagedBatch in the forms that its callers choose from: streams given by object and by handle, several streams,
4 bits, masks, weights per head, the default output, merging."""
import math

import numpy as np
import pytest

from test_gpu_paged import SPECS, ctx_of, ints, rows

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qwm():
    import bit_kv_cache_qsac_gb300 as q
    return q


def batch_of(qwm, H, kv, layers=1, **kw):
    from bit_kv_cache_qsac_gb300.stream import PagedBatch
    kw = dict(dict(batch=4, max_tokens=300, pages=60, rows=120, page=16, rope=qwm.RopeSpec(**SPECS["text"])), **kw)
    return PagedBatch(ctx_of(qwm, H), layers, kv, **kw)


def inputs(rng, H, kv, n):
    return rows(rng, H, n), rows(rng, kv, n), rows(rng, kv, n)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("norm", [True, False])
def test_a_stream_by_object_and_by_handle(qwm, norm, handle):
    rng, H, kv = np.random.default_rng(1), 4, 2
    one, two = (batch_of(qwm, H, kv, norm=norm) for _ in range(2))
    count, (q, k, v) = ints([50, 1, 0, 60], torch.int32), inputs(rng, H, kv, 120)
    one.begin(count)
    want = one.layer(0, q, k, v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = side.cuda_stream if handle else side
    two.begin(count, stream=s)
    got = two.layer(0, q, k, v, stream=s)
    side.synchronize()
    assert torch.equal(got, want) and bool(got.any())


def test_calls_on_several_streams_follow_one_another(qwm):
    """A batch built behind long work on its stream, its steps begun on a second one and its layers called on others: each
    call finds what those before it left (an earlier one is held up by spinning, half a second in all)."""
    rng, H, kv = np.random.default_rng(2), 4, 2
    counts = [ints(c, torch.int32) for c in ([60, 1, 20, 0], [1, 1, 1, 90], [2, 30, 1, 1])]
    keeps = [ints(k) for k in ([1 << 40] * 4, [40, 1 << 40, 1 << 40, 1 << 40], [1 << 40, 0, 1 << 40, 80])]
    steps = [[inputs(rng, H, kv, 120) for _ in range(2)] for _ in counts]

    def run(pb, streams, hold):
        out = []
        for i, (c, k) in enumerate(zip(counts, keeps)):
            hold(streams[i % 4])
            granted = pb.begin(c, k, stream=streams[i % 4])
            for j, (q, kk, v) in enumerate(steps[i]):
                hold(streams[(i + j + 1) % 4])
                o = torch.zeros(120, H, 128, dtype=torch.bfloat16, device="cuda").permute(1, 0, 2)
                torch.cuda.current_stream().synchronize()   # the output is there; what the batch does is its own to order
                out.append(pb.layer(j, q, kk, v, out=o, stream=streams[(i + j + 1) % 4]))
        torch.cuda.synchronize()
        return out, granted.tolist(), pb.table.length.tolist()
    main = torch.cuda.current_stream()
    want = run(batch_of(qwm, H, kv, layers=2), [main] * 4, lambda s: None)
    torch.cuda.synchronize()

    def hold(s):
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)   # some 10 ms
    side = [torch.cuda.Stream() for _ in range(4)]
    built = torch.cuda.Stream()
    hold(built)
    with torch.cuda.stream(built):
        pb = batch_of(qwm, H, kv, layers=2)
    got = run(pb, side, hold)
    assert got[1:] == want[1:] and pb.check() == qwm.QWM_OK
    assert all(torch.equal(a, b) for a, b in zip(got[0], want[0])) and bool(got[0][0].any())


@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("known", [False, True])      # max_count given: other kernels, or the same
@pytest.mark.parametrize("given", ["none", "fp32", "bf16"])
@pytest.mark.parametrize("bits,mask,weights,norm,rope", [
    (4, dict(tpf=1, frames=30, sink=5), "heads", True, "text"), (8, dict(tpf=16, frames=2, sink=16), "one", True, "video"),
    (4, dict(), "heads", True, None), (4, dict(tpf=1, frames=64, sink=0), None, False, "video"), (8, dict(tpf=10, frames=3, sink=4), None, True, "text")])
def test_paged_batch_is_its_calls(qwm, bits, mask, weights, norm, rope, given, known, side):
    """A step of PagedBatch is, bit for bit, the calls that the header names, made one after the other: at both widths,
    under windows with sinks and frames, with weights per head, into the default output (whose padding rows are 0) and
    given ones, merged into an earlier result, with the largest count known or not, on a stream of its own."""
    rng, H, kv, n, page = np.random.default_rng(bits + len(mask)), 6, 2, 120, 16
    kw = SPECS[rope] if rope else None
    spec = qwm.RopeSpec(**kw) if rope else None
    pb = batch_of(qwm, H, kv, layers=2, bits=bits, norm=norm, rope=spec, **mask)
    ctx = pb.ctx
    w = {"heads": lambda h: (h, 128), "one": lambda h: (128,), None: None}[weights]
    wq, wk = (torch.from_numpy(rng.uniform(0.5, 1.5, w(h)).astype(np.float32)).cuda() if w else None for h in (H, kv))
    tab, pools = qwm.PageTable.empty(4, -(-300 // page), page, 60), [qwm.PagePool.empty(bits, page, 60, kv) for _ in range(2)]
    first, granted = (torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(2))
    slot, at = (torch.full((n,), -1, dtype=torch.int64, device="cuda") for _ in range(2))
    stream = torch.cuda.Stream() if side else None
    for counts in ([50, 3, 0, 40], [1, 1, 1, 90], [1, 4, 2, 1]):
        count = ints(counts, torch.int32)
        layers = [inputs(rng, H, kv, n) for _ in range(2)]
        earlier = [(torch.randn(H, n, 128, device="cuda"), torch.randn(H, n, device="cuda")) for _ in range(2)]
        torch.cuda.synchronize()
        assert pb.begin(count, stream=stream) is pb.granted
        got = []
        for i, (q, k, v) in enumerate(layers):
            out, lse = None, None
            if given == "fp32":
                out, lse = earlier[i][0].clone(), earlier[i][1].clone()
            elif given == "bf16":
                out, lse = torch.full((H, n, 128), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((H, n), 3.0, device="cuda")
            torch.cuda.synchronize()
            o = pb.layer(i, q, k, v, wq, wk, out=out, lse=lse, merge=given == "fp32", max_count=max(counts) if known else None, stream=stream)
            assert out is None or o is out
            got.append((o, lse))
        torch.cuda.synchronize()
        qwm.qwm_pages_update(ctx, tab, first, granted, slot, at, count=count)
        assert granted.tolist() == counts == pb.granted.tolist()
        live = sum(counts)
        for i, (q, k, v) in enumerate(layers):
            qwm.qwm_paged_write(ctx, pools[i], k, v, slot, at=at if rope else None, rope=spec, norm=norm, weight=wk, eps=1e-6)
            ready = q.clone()
            if norm:
                qwm.qwm_norm_rope(ctx, spec, q[None], wq, 1e-6, ready[None], at=at[None] if rope else None)
            elif rope:
                p = at.clamp(min=0)   # (padding rows are not attended with)
                pos = torch.stack([p // math.prod(kw["grid"]), p // kw["grid"][1] % kw["grid"][0], p % kw["grid"][1]], -1).to(torch.int32)
                qwm.qwm_rope(ctx, spec, q[None], ints([0]), ready[None], pos=pos[None])
            want = torch.zeros(H, n, 128, dtype=torch.bfloat16, device="cuda")
            wl = torch.zeros(H, n, device="cuda")
            if given == "fp32":
                want, wl = earlier[i][0].clone(), earlier[i][1].clone()
            elif given == "bf16":
                want.fill_(3.0), wl.fill_(3.0)
            qwm.qwm_paged_attend(ctx, pools[i], tab, ready, first, granted, 128 ** -0.5, want, lse=wl, merge=given == "fp32",
                                 max_count=max(counts) if known else n, **mask)
            o, lse = got[i]
            assert o.dtype == want.dtype and torch.equal(o, want) and (lse is None or torch.equal(lse, wl))
            if given == "none":
                assert not o[:, live:].any() and bool(o[:, :live].any())
            for t in ("k_codes", "k_step", "v_codes", "v_step"):
                assert torch.equal(getattr(pb.pools[i], t), getattr(pools[i], t))
    assert pb.check() == qwm.QWM_OK


def test_tokens_go_on_to_be_packed(qwm):
    """The hand-over that the paged cache is made for: tokens of a sequence read back in bf16, in order of their
    positions, are packed as history and attended there; the result is that of the same rows packed directly."""
    from bit_kv_cache_qsac_gb300.stream import CompressedLayer
    rng, H, n = np.random.default_rng(9), 4, 256
    ctx, pb = ctx_of(qwm, H), batch_of(qwm, H, H, rows=n, pages=40, max_tokens=512)
    q, k, v = inputs(rng, H, H, n)
    pb.begin(ints([0, n, 0, 0], torch.int32))
    pb.layer(0, q, k, v)
    t = torch.arange(n, device="cuda")
    slots = pb.table.table[1].long()[t // 16] * 16 + t % 16
    assert torch.equal(slots, pb.slot)
    hats = [torch.empty(H, n, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    qwm.qwm_paged_read(ctx, pb.pools[0], slots, *hats)
    pb.begin(ints([0] * 4, torch.int32), ints([0] * 4))   # the pages are free again
    assert int(pb.table.free_count) == 40
    layer = CompressedLayer(ctx)
    layer.append_chunk(*hats)
    out = layer.attend(q.contiguous())
    kh, vh = layer.dequantize(0)
    assert pb.check() == qwm.QWM_OK
    x = torch.softmax(q.double() @ kh.double().transpose(1, 2) / math.sqrt(128), -1) @ vh.double()
    # the history's attention against its own dequantised rows (bf16 here, 2^-8 of Keys' logits and of Values)
    mag = (q.double().abs() @ kh.double().abs().transpose(1, 2)).amax(-1, keepdim=True) / math.sqrt(128)
    assert bool(((out.double() - x).abs() <= (2 * 2.0 ** -8 * mag + 2.0 ** -7) * vh.double().abs().amax()).all())
    # and they stand for what came, within the 2-bit packing: an order of rows or heads mixed up would not
    for hat, packed in ((hats[0], kh), (hats[1], vh)):
        own = (packed.double() - hat.double()).norm() / hat.double().norm()
        other = (packed.double().roll(1, 1) - hat.double()).norm() / hat.double().norm()
        assert float(own) < 0.5 * float(other)
