"""The fp32 losses' errors in the norm (loss_accuracy.py): on the GPU, and on the
host the check itself against planes that are missing."""
import pytest
import torch

from tests import loss_accuracy as acc
from tests import loss_reference as ref

SHAPES = [(33, 1031, 200), (64, 2000, 512), (300, 1500, 96), (130, 700, 1000)]


def planes(x, count):
    """x as `count` bf16 planes, in float64."""
    out, x = [], x.double()
    for _ in range(count):
        out.append(x.float().bfloat16().double())
        x = x - out[-1]
    return out


def by_planes(count):
    """Products of operands in `count` planes, those terms kept that are above the last plane's size."""
    def product(a, b):
        pa, pb = planes(a, count), planes(b, count)
        return sum(pa[i] @ pb[j].t() for i in range(count) for j in range(count - i))
    return product


@pytest.mark.parametrize("T,V,D", SHAPES)
def test_the_check_accepts_three_planes_and_rejects_two(T, V, D):
    h, w, y, g = acc.operands(T, V, D, "cpu")
    want = acc.definition(h, w, y, g)
    acc.check(want, acc.definition(h, w, y, g, by_planes(3)))
    two = acc.definition(h, w, y, g, by_planes(2))
    for name in ("dh", "dw"):
        with pytest.raises(AssertionError, match=name):
            acc.check(want, {name: two[name]})


@pytest.mark.parametrize("T,V,D", SHAPES)
def test_the_definition_is_the_reference_s(T, V, D):
    h, w, y, g = acc.operands(T, V, D, "cpu")
    r = ref.xent(h, w, y, g=g)
    for name, x in acc.definition(h, w, y, g).items():
        assert torch.allclose(x, getattr(r, name), rtol=1e-12, atol=1e-14), name


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,D", SHAPES + [(5, 4096, 1024), (16, 16384, 300), (40, 3000, 4096), (300, 4096, 1024),
                                            (600, 1031, 513), (2000, 1500, 512), (33, 20000, 64), (700, 900, 2100)])
def test_fp32_errors_in_the_norm(T, V, D):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from tests import gpu_harness as H
    lib = H.tg()
    h, w, y, g = acc.operands(T, V, D, "cuda")
    loss, lse = lib.linear_cross_entropy(h, w, y)
    dh, dw = lib.linear_cross_entropy_backward(h, w, y, lse, g)
    assert lib.device_status(torch.cuda.current_stream().cuda_stream) == lib.OK
    acc.check(acc.definition(h, w, y, g), {"loss": loss, "lse": lse, "dh": dh, "dw": dw})


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 40, 300])
def test_fp32_distillation_errors_in_the_norm(T):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from tests import gpu_harness as H
    lib = H.tg()
    h, w, _, g = acc.operands(T, 1500, 700, "cuda")
    ids = torch.randint(0, 1500, (T, 9), device="cuda")
    logits = torch.randn(T, 9, device="cuda")
    loss, lse = lib.linear_distillation(h, w, ids, logits)
    dh, dw = lib.linear_distillation_backward(h, w, ids, logits, lse, g)
    r = ref.distill(h, w, ids, logits, 1.0, g)
    acc.check({n: getattr(r, n) for n in ("loss", "lse", "dh", "dw")}, {"loss": loss, "lse": lse, "dh": dh, "dw": dw})


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("T,counting,most", [(2, 2, 1.05), (20, 20, 1.05), (32, 7, 1.05), (33, 33, 1.6), (300, 300, 1.6),
                                             (300, 2, 2.7)])
def test_16_bit_gradients_beside_their_own_rounding(T, counting, most, dtype):
    """dH and dW against the exact ones, in units of what their last rounding alone leaves, in the norm.  Up to 32 rows
    dz has two planes (or is fp32) and adds nothing to it.  Above, dz is rounded to the type too: a rounding of the same
    size, independent of the last, makes sqrt(2), and a tenth more is left for its spread.  With two rows that
    count, a gradient may hang on one entry of dz, whose rounding is up to 2.4 times an average one: sqrt(1 + 2.4^2)."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from tests import gpu_harness as H
    lib = H.tg()
    V, D = 4096, 512
    h, w, y, g = acc.operands(T, V, D, "cuda", seed=T)
    h, w, g = h.to(dtype), (2 * w).to(dtype), 0.5 + g
    alone = (h[:counting], w, y[:counting], g[:counting])
    y = y.clone()
    y[counting:] = -100
    loss, lse = lib.linear_cross_entropy(h, w, y)
    dh, dw = lib.linear_cross_entropy_backward(h, w, y, lse, g)
    assert lib.device_status(torch.cuda.current_stream().cuda_stream) == lib.OK
    want = acc.definition(*alone)
    for got, exact in ((dh[:counting], want["dh"]), (dw, want["dw"])):
        own = (exact.to(dtype).double() - exact).norm()
        assert float((got.double() - exact).norm() / own) <= most
