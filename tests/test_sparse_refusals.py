"""Refusals of routing through the C ABI, each call by itself: the status of both directions.  No call reaches the GPU."""
import pytest

A0, B0, C0, D0, E0 = (0x1000000000 * (i + 1) for i in range(5))


@pytest.fixture(scope="module")
def tg():
    from tests.conftest import build_library
    build_library()
    import tiled_dense_gemm_02_gb300 as tg
    return tg


@pytest.mark.parametrize("E,k,more,status", [(1024, 4, {}, "OK"), (1025, 4, {}, "ERR_TOO_LARGE"), (1 << 20, 4, {}, "ERR_TOO_LARGE"),
                                             (64, 33, {}, "ERR_TOO_LARGE"), (64, 4, {"groups": 64}, "ERR_TOO_LARGE"),
                                             (64, 65, {}, "ERR_INVALID_VALUE"), (64, 4, {"groups": 3}, "ERR_INVALID_VALUE")])
def test_sizes_past_the_limits(tg, E, k, more, status):
    """T = 0 ends a call that is accepted before it looks at the device."""
    want = getattr(tg, status)
    assert tg.route_forward(0, E, k, A0, E, 2, B0, C0, D0, more or None) == want
    assert tg.route_backward(0, E, k, A0, E, 2, C0, D0, E0, E, more or None) == want
