"""examples/train_sparse_layer.py runs, and its step's gradients are those of the definition."""
import importlib.util
import math
import os

import pytest
import torch

from tests import gpu_harness as H
from tests.experts_reference import Experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    H.tg()
    torch.cuda.set_device(0)
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_sparse_layer.py")
    spec = importlib.util.spec_from_file_location("train_sparse_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_it_runs(example):
    for dtype in (torch.bfloat16, torch.float16):
        history = example.train(tokens=300, depth=64, width=48, experts=6, steps=3, dtype=dtype)
        assert len(history) == 3 and all(math.isfinite(v) for row in history for v in row)


def test_its_gradients(example):
    lib = H.tg()
    gen = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen).bfloat16()

    hidden, router, target = normal(200, 64), normal(6, 64) * 0.1, normal(200, 64).float()
    w_in, w_out = normal(6, 96, 64) / 8, normal(6, 64, 48) / 7
    bias = torch.zeros(6, device="cuda")
    loss, norm, ids, (d_router, d_in, d_out) = example.step(hidden, target, router, w_in, w_out, bias, 2, 1e9)
    logits = lib.matmul(hidden, router.t().contiguous(), out_dtype=torch.float32)
    picks, weights = lib.route_experts(logits, 2, scoring="sigmoid", bias=bias)
    assert torch.equal(ids, picks)
    out, saved = lib.expert_mlp(hidden, w_in, w_out, ids, weights, save=True)
    error = out.float() - target
    assert float(loss) == float(error.square().mean())
    grad = (error * (2.0 / error.numel())).bfloat16()
    Experts(hidden, w_in, w_out, ids, weights, grad).check(dw_in=d_in, dw_out=d_out)
    d_weights = lib.expert_mlp_backward(hidden, w_in, w_out, ids, weights, saved, grad)[3]
    d_logits = lib.route_experts_backward(logits, ids, d_weights, scoring="sigmoid").bfloat16().double()
    want, size = d_logits.t() @ hidden.double(), d_logits.abs().t() @ hidden.double().abs()
    assert bool(((d_router.double() - want).abs() <= 2.0 ** -10 * size).all())
    whole = math.sqrt(sum(float(g.double().square().sum()) for g in (d_router, d_in, d_out)))
    assert abs(float(norm) - whole) <= 18 * 2.0 ** -24 * whole
    clipped = example.step(hidden, target, router, w_in, w_out, bias, 2, whole / 2)[3]
    for a, b in zip(clipped, (d_router, d_in, d_out)):
        # half, the factor's and the product's roundings, and one of the type's
        assert bool(((a.double() - b.double() / 2).abs() <= b.double().abs() / 2 * (20 * 2.0 ** -24 + torch.finfo(a.dtype).eps / 2)).all())
