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


def test_options_held_in_tensors_are_read_at_every_call(tg):
    """A weight kept in a tensor and changed in place (a schedule) is the value that the next call uses."""
    import torch
    from tiled_dense_gemm_02_gb300 import loss
    z, eps, scale = torch.tensor(1e-4), torch.tensor(0.0), torch.tensor(2.0)
    first = loss._options(*loss._plain(scale, eps, z, 0, -100))._obj
    z.fill_(0.5)
    eps.fill_(0.25)
    scale.fill_(4.0)
    then = loss._options(*loss._plain(scale, eps, z, 0, -100))._obj
    assert (first.scale, first.label_smoothing, first.z_loss) == (2.0, 0.0, pytest.approx(1e-4))
    assert (then.scale, then.label_smoothing, then.z_loss) == (4.0, 0.25, 0.5)


def test_tensor_functions_pass_options_as_plain_numbers(tg, monkeypatch):
    import torch
    from tiled_dense_gemm_02_gb300 import loss
    seen = []

    def options(*values):
        seen.append(values)
        raise KeyError  # far enough

    monkeypatch.setattr(loss, "_options", options)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    h, w, y, ids, logits, g = on_no_device()
    more = {"label_smoothing": torch.tensor(0.25), "z_loss": torch.tensor(0.5), "scale": torch.tensor(2.0),
            "ignore_index": torch.tensor(7), "piece": torch.tensor(256)}
    for call in (lambda: tg.linear_cross_entropy(h, w, y, **more),
                 lambda: tg.linear_cross_entropy_backward(h, w, y, g, g, **more),
                 lambda: tg.linear_distillation(h, w, ids, logits, temperature=torch.tensor(0.5),
                                                piece=torch.tensor(256))):
        with pytest.raises(KeyError):
            call()
    assert seen[0] == seen[1] == (2.0, 0.25, 0.5, 256, 7) and seen[2] == (2.0, 0.0, 0.0, 256, 0)
    for values in seen:
        assert [type(v) for v in values] == [float, float, float, int, int]
