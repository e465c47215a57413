"""What the tensor functions of the vocabulary-head losses hand to the library
as options, on the host: no call here reaches the GPU."""
import pytest


@pytest.fixture(scope="module")
def tg():
    from tests.conftest import build_library
    build_library()
    import tiled_dense_gemm_02_gb300 as tg
    return tg


def on_no_device(T=4, V=10, D=8, K=3):
    import torch
    h, w = torch.zeros(T, D, dtype=torch.bfloat16), torch.zeros(V, D, dtype=torch.bfloat16)
    return h, w, torch.zeros(T, dtype=torch.int64), torch.zeros(T, K, dtype=torch.int64), torch.zeros(T, K), torch.ones(T)


@pytest.mark.parametrize("scale", [1e-46, 1e-300, float("inf"), 1e39, float("nan"), 0.0, -1.0])
def test_scales_that_fp32_does_not_hold_are_refused(tg, scale):
    """The library reads a scale of 0 as its default, 1: one that rounds to 0 must not get there."""
    h, w, y, _, _, g = on_no_device()
    for call in (lambda: tg.linear_cross_entropy(h, w, y, scale=scale),
                 lambda: tg.linear_cross_entropy_backward(h, w, y, g, g, scale=scale)):
        with pytest.raises(ValueError, match="scale"):
            call()


@pytest.mark.parametrize("temperature", [float("inf"), 1e46, 1e300, 1e-39, 1e-320, float("nan"), 0.0, -1.0])
def test_temperatures_whose_reciprocal_fp32_does_not_hold_are_refused(tg, temperature):
    h, w, _, ids, logits, g = on_no_device()
    for call in (lambda: tg.linear_distillation(h, w, ids, logits, temperature=temperature),
                 lambda: tg.linear_distillation_backward(h, w, ids, logits, g, g, temperature=temperature)):
        with pytest.raises(ValueError, match="temperature"):
            call()


def test_scales_that_fp32_holds_reach_the_device_check(tg):
    h, w, y, ids, logits, _ = on_no_device()
    for scale in (1e-44, 1e-30, 0.5, 1e38):
        with pytest.raises(ValueError, match="CUDA device"):
            tg.linear_cross_entropy(h, w, y, scale=scale)
        with pytest.raises(ValueError, match="CUDA device"):
            tg.linear_distillation(h, w, ids, logits, temperature=1 / scale)
