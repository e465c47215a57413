"""Clipping where the norm is at or past fp32's largest number: what the norm says is what was done."""
import math

import pytest
import torch

from tests import gpu_harness as H

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    H.tg()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype,n,value", [(F32, 2, 3e38), (F32, 5000, 1e38), (BF16, 40_000, 2e38), (F32, 1_000_000, 3.4e38)])
def test_a_norm_past_fp32_scales_nothing(dtype, n, value):
    """The norm is finite in 64 bits and infinite as it is returned: nothing is scaled, in place or not."""
    lib = H.tg()
    grads = [torch.full((n,), value, device="cuda").to(dtype), torch.ones(33, device="cuda")]
    kept = [g.clone() for g in grads]
    out = [torch.full_like(g, 7.0) for g in grads]
    assert float(lib.clip_gradients(grads, 1.0, outputs=out)) == math.inf
    assert float(lib.clip_gradients(grads, 1.0)) == math.inf
    for a, b, c in zip(grads, out, kept):
        assert torch.equal(a, c) and torch.equal(b, c)


def test_a_norm_just_below_the_largest_number_scales():
    lib = H.tg()
    top = torch.finfo(F32).max
    for value, scales in ((top, True), (top * (1 - 2.0 ** -20), True)):
        g = torch.zeros(100, device="cuda")
        g[17] = value
        norm = float(lib.clip_gradients([g], 1e30))
        assert norm == float(torch.tensor(value, dtype=F32))
        # factor, product and the norm's rounding: 2^-24 each, and the square's 2^-24
        assert abs(float(g[17]) / 1e30 - 1.0) <= 5 * 2.0 ** -24
