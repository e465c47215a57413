"""Numbers at the ends of their range in the vocabulary-head losses: where a
computation that is right in the middle of it overflows, underflows or is moved."""
import math

import pytest
import torch

from tests import gpu_harness as H
from tests import loss_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    H.tg()
    torch.cuda.set_device(0)


def head(T, V, D, dtype, seed=0, spread=2.0):
    gen = torch.Generator(device="cuda").manual_seed(7000 + seed)
    h = torch.randn(T, D, device="cuda", generator=gen).to(dtype)
    w = (torch.randn(V, D, device="cuda", generator=gen) * (spread / math.sqrt(D))).to(dtype)
    return h, w, gen


def finished():
    lib = H.tg()
    assert lib.device_status(torch.cuda.current_stream().cuda_stream) == lib.OK


@pytest.mark.parametrize("logits_dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [6, 300])
def test_teacher_logits_whose_multiples_leave_the_range(T, logits_dtype):
    """Rows of the type's lowest value alone are uniform at any temperature, and a large top has all the mass."""
    lib = H.tg()
    V, D, K = 900, 64, 6
    h, w, gen = head(T, V, D, BF16)
    ids = torch.randint(0, V, (T, K), device="cuda", generator=gen)
    logits = (4 * torch.randn(T, K, device="cuda", generator=gen)).to(logits_dtype)
    low, top = torch.finfo(logits_dtype).min, torch.finfo(logits_dtype).max
    logits[1] = low
    logits[2] = low
    logits[2, 3] = 1.0
    logits[3] = top
    logits[4, 2:] = low
    logits[4, :2] = 0.75 * top
    logits[5] = float("-inf")
    logits[5, 1:3] = low
    g = torch.rand(T, device="cuda", generator=gen)
    for temperature in (0.25, 1.0, 3.0):
        loss, lse = lib.linear_distillation(h, w, ids, logits, temperature=temperature)
        dh, dw = lib.linear_distillation_backward(h, w, ids, logits, lse, g, temperature=temperature)
        finished()
        ref.distill(h, w, ids, logits, temperature, g).check(loss=loss, lse=lse, dh=dh, dw=dw)
