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
