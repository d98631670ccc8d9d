"""Host-side limits of the recent window (no GPU)."""
import pytest

import window_ref as ref


@pytest.fixture(scope="module")
def qwm():
    import __graft_entry__
    __graft_entry__.build_library()
    import bit_kv_cache_qsac_gb300 as q
    return q


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("theta", [1.0, 2.0, 256.0, 1e4, 123456.789, 5e5, 1e300, (1e4, 1e3, 50.0)])
@pytest.mark.parametrize("dims", [(128, 0, 0), (44, 42, 42), (2, 4, 30)])
def test_plan_turns_are_rounded_once(qwm, dims, theta, shared, inverse):
    """Each entry is the exact part of a turn to half a unit of 2^-64 (2^-20 of a unit for the arithmetic of
    some 100 bits): positions multiply what is left."""
    spec = qwm.RopeSpec(dims, theta=theta, shared_freq=shared, inverse=inverse)
    exact = ref.exact_turns(dims, theta if isinstance(theta, tuple) else (theta,) * 3, shared)
    for i, t in enumerate(exact):
        got = spec.turn[i] if not inverse else -spec.turn[i] % 2 ** 64
        assert abs(got * 2 ** 136 - t) <= 2 ** 135 + 2 ** 116, (i, got, t / 2 ** 136)
