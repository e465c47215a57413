"""The experts' products on the GPU against their definition in 64 bits
(tests/experts_reference.py), at the sizes, lists and layouts where they can go
wrong, through the tensor functions and through the C ABI."""
import math

import pytest
import torch

from tests import gpu_harness as H
from tests.experts_reference import Experts

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
NAMES = {BF16: "bf16", F16: "f16"}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    H.tg()
    torch.cuda.set_device(0)


def layer(T, E, k, D, F, dtype, seed=0, pad=0, skew=0.5):
    gen = torch.Generator(device="cuda").manual_seed(2000 + seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    x = normal(T, D + pad).to(dtype)[:, :D]
    w_in = (normal(E, 2 * F, D) / math.sqrt(D)).to(dtype)
    w_out = (normal(E, D, F) / math.sqrt(F)).to(dtype)
    ids = torch.topk(normal(T, E) + skew * normal(E), k, dim=1).indices
    weights = torch.rand(T, k, device="cuda", generator=gen)
    return x, w_in, w_out, ids, weights, (0.1 * normal(T, D)).to(dtype), gen


def finished():
    lib = H.tg()
    assert lib.device_status(torch.cuda.current_stream().cuda_stream) == lib.OK
    return lib


def both(x, w_in, w_out, ids, weights, g, **more):
    lib = H.tg()
    plain, none = lib.expert_mlp(x, w_in, w_out, ids, weights)
    assert none is None
    out, saved = lib.expert_mlp(x, w_in, w_out, ids, weights, save=True)
    dx, dw_in, dw_out, dw = lib.expert_mlp_backward(x, w_in, w_out, ids, weights, saved, g, **more)
    finished()
    return plain, {"out": out, "dx": dx, "dw_in": dw_in, "dw_out": dw_out, "dw": dw}


def check(x, w_in, w_out, ids, weights, g):
    plain, got = both(x, w_in, w_out, ids, weights, g)
    Experts(x, w_in, w_out, ids, weights, g).check(**got)
    Experts(x, w_in, w_out, ids, weights).check(out=plain)
    return got


SHAPES = [(1, 1, 1, 8, 8), (1, 4, 2, 64, 64), (2, 3, 3, 1, 1), (3, 5, 2, 72, 40), (7, 2, 1, 65, 33), (17, 8, 4, 128, 256),
          (33, 4, 2, 200, 136), (64, 16, 8, 256, 128), (100, 3, 2, 130, 250), (129, 2, 2, 512, 64), (256, 8, 2, 192, 384),
          (257, 1, 1, 264, 72), (300, 6, 3, 520, 520), (513, 4, 2, 100, 700), (700, 2, 1, 640, 272), (1000, 10, 3, 331, 170),
          (31, 200, 5, 64, 24)]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=NAMES.get)
@pytest.mark.parametrize("T,E,k,D,F", SHAPES)
def test_forward_and_backward_match_the_definition(T, E, k, D, F, dtype):
    check(*layer(T, E, k, D, F, dtype, seed=T + D)[:6])
