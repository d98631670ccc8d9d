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
