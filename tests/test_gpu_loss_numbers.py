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


def masked_head(T, V, D, dtype, seed):
    """A column of ones in H against one of 0 and -inf in W: every third entry, target aside, is masked out.
    Returns H, W, the targets, and W and the targets with the masked entries left out."""
    h, w, gen = head(T, V, D, dtype, seed)
    h[:, D - 1] = 1.0
    keep = torch.arange(V, device="cuda") % 3 != 1
    w[:, D - 1] = 0.0
    w[~keep, D - 1] = float("-inf")
    kept = torch.nonzero(keep)[:, 0]
    at = torch.randint(0, kept.numel(), (T,), device="cuda", generator=gen)
    return h, w, kept[at], w[keep], at


@pytest.mark.parametrize("T,V,D,dtype", [(1, 1000, 64, BF16), (1, 777, 37, F16), (3, 777, 41, BF16), (8, 900, 50, F16),
                                         (5, 900, 64, F32), (16, 16384, 40, F32), (16, 900, 40, F32), (64, 900, 128, BF16),
                                         (300, 2000, 600, F16)])
def test_entries_masked_by_an_infinite_logit(T, V, D, dtype):
    lib = H.tg()
    h, w, y, w_kept, y_kept = masked_head(T, V, D, dtype, T + V)
    loss, lse = lib.linear_cross_entropy(h, w, y)
    finished()
    ref.xent(h, w_kept, y_kept).check(loss=loss, lse=lse)
    ids, logits = y[:, None].expand(T, 2).contiguous(), torch.randn(T, 2, device="cuda")
    loss, lse = lib.linear_distillation(h, w, ids, logits)
    finished()
    ref.distill(h, w_kept, y_kept[:, None].expand(T, 2).contiguous(), logits).check(loss=loss, lse=lse)


@pytest.mark.parametrize("T,V,D,dtype", [(1, 1000, 64, BF16), (2, 777, 40, F16), (3, 777, 41, BF16), (5, 900, 64, F32),
                                         (16, 16384, 40, F32), (33, 900, 40, F32), (64, 900, 128, BF16),
                                         (300, 2000, 600, F16), (300, 1000, 70, F32)])
def test_entries_masked_by_the_lowest_value(T, V, D, dtype):
    """The type's lowest value, which no sum of logits moves: no mass, no gradient, and none of it in the others'."""
    lib = H.tg()
    h, w, y, w_kept, y_kept = masked_head(T, V, D, dtype, T + V)
    masked = torch.isinf(w[:, D - 1])
    w[masked, D - 1] = torch.finfo(dtype).min
    g = torch.rand(T, device="cuda")
    loss, lse = lib.linear_cross_entropy(h, w, y)
    dh, dw = lib.linear_cross_entropy_backward(h, w, y, lse, g)
    finished()
    assert bool((dw[masked] == 0).all())
    ref.xent(h, w_kept, y_kept, g=g).check(loss=loss, lse=lse, dh=dh, dw=dw[~masked])


@pytest.mark.parametrize("T", [5, 20, 200])
@pytest.mark.parametrize("kind", ["xent", "distill"])
def test_fp16_rows_of_small_weight_beside_large_ones(kind, T):
    """A flat softmax over a large vocabulary whose weights share a mean: the softmax's part of dH is a sum of V equal
    terms, so a probability that falls out of fp16's range is seen whole."""
    lib = H.tg()
    V, D = 100000, 64
    h, w, gen = head(T, V, D, F16, spread=0.5)
    h *= 0.125
    w += torch.randn(D, device="cuda", generator=gen).to(F16)
    y = torch.randint(0, V, (T,), device="cuda", generator=gen)
    sizes = torch.tensor([1.0, 1e-1, 1e-2, 1e-3, 1e-4, 1e-5, 1e-6, 3e-7], device="cuda")
    g = 2000.0 * sizes[torch.arange(T, device="cuda") % 8] * (0.5 + 0.5 * torch.rand(T, device="cuda", generator=gen))
    g[4] = -g[4]
    if kind == "xent":
        more = {"label_smoothing": 0.1, "z_loss": 1e-3}
        loss, lse = lib.linear_cross_entropy(h, w, y, **more)
        dh, dw = lib.linear_cross_entropy_backward(h, w, y, lse, g, **more)
        r = ref.xent(h, w, y, smoothing=0.1, z_loss=1e-3, g=g)
    else:
        ids = torch.randint(0, V, (T, 7), device="cuda", generator=gen)
        logits = torch.randn(T, 7, device="cuda", generator=gen)
        loss, lse = lib.linear_distillation(h, w, ids, logits)
        dh, dw = lib.linear_distillation_backward(h, w, ids, logits, lse, g)
        r = ref.distill(h, w, ids, logits, 1.0, g)
    finished()
    r.check(loss=loss, lse=lse, dh=dh, dw=dw)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("D", [512, 4096, 16384])
def test_logits_whose_sums_are_exact(D, T, dtype):
    """One-hot hidden states and weights of few bits: every partial sum is a number that fp32 holds, so nothing may move
    a logit.  What is left are the roundings of the exponentials (2^-22 each, one way), of their sum and logarithm
    and of the last sums: 2^-20 (1 + |lse|) in all, as in the tests' reference; a logit of 20 moved by 4e-6
    of itself is four times that off."""
    lib = H.tg()
    V = 700
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    h = torch.zeros(T, D, device="cuda", dtype=dtype)
    at = torch.randint(0, D, (T,), device="cuda", generator=gen)
    h[torch.arange(T, device="cuda"), at] = 16.0
    w = torch.randint(-2, 3, (V, D), device="cuda", generator=gen).to(dtype) / 4
    y = torch.randint(0, V, (T,), device="cuda", generator=gen)
    w[y] += 0.75  # the targets' logits: up to 20
    loss, lse = lib.linear_cross_entropy(h, w, y)
    finished()
    z = h.double() @ w.double().t()
    want = torch.logsumexp(z, dim=1)
    bound = 2.0 ** -20 * (1 + want.abs())
    assert bool(((lse.double() - want).abs() <= bound).all())
    exact = want - z.gather(1, y[:, None])[:, 0]
    assert bool(((loss.double() - exact).abs() <= 2 * bound).all())


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("D", [4096, 32768])
def test_logits_of_products_of_one_sign(D, T, dtype):
    """All products positive: the sums grow with every step, and so would the losses of an adder that truncates.  At most
    64 steps of 16 products truncate one sum, each by less than 2^-23 of it, before it is added to the others with
    rounding to nearest (2^-24 an addition, one for 1024 or fewer products): the bound does not grow with D but by these."""
    lib = H.tg()
    V = 600
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    h = torch.rand(T, D, device="cuda", generator=gen).to(dtype)
    w = (torch.rand(V, D, device="cuda", generator=gen) * (80.0 / D)).to(dtype)  # logits of about 20
    y = torch.randint(0, V, (T,), device="cuda", generator=gen)
    loss, lse = lib.linear_cross_entropy(h, w, y)
    finished()
    z = h.double() @ w.double().t()
    want = torch.logsumexp(z, dim=1)
    e_z = (64 * 2.0 ** -23 + D / 512 * 2.0 ** -24) * z.amax(dim=1)
    bound = e_z + 2.0 ** -20 * (1 + want.abs())
    assert bool(((lse.double() - want).abs() <= bound).all()), float(((lse.double() - want).abs() / bound).max())
    # a common factor of all logits cancels in the loss but for their differences
    exact = want - z.gather(1, y[:, None])[:, 0]
    assert bool(((loss.double() - exact).abs() <= 2 * bound).all())


def mean_error(got, want):
    return float(((got.double() - want) / want).mean())


def test_gradient_sums_of_one_sign_over_long_axes():
    """fp16 gradients whose terms have one sign and are exact: their mean error is what the adder's truncation leaves.
    256 steps of less than 2^-23 of the sum each are 2^-15; the rounding to fp16 (2^-11 at most, both ways) leaves four
    of its deviations, 2^-11 / sqrt(3 n), in the mean of n values."""
    lib = H.tg()
    gen = torch.Generator(device="cuda").manual_seed(11)

    def bound(n):
        return 2.0 ** -15 + 4 * 2.0 ** -11 / math.sqrt(3 * n)

    # dW: W = 0, so every probability is 2^-8; 65536 rows of positive h with one target
    T, V, D = 65536, 256, 1024
    h = (0.5 + 0.5 * torch.rand(T, D, device="cuda", generator=gen)).to(F16)
    w = torch.zeros(V, D, device="cuda", dtype=F16)
    y = torch.zeros(T, device="cuda", dtype=torch.int64)
    g = torch.ones(T, device="cuda")
    _, lse = lib.linear_cross_entropy(h, w, y)
    _, dw = lib.linear_cross_entropy_backward(h, w, y, lse, g, want_hidden=False)
    finished()
    assert abs(mean_error(dw[7], h.double().sum(dim=0) / V)) <= bound(D)
    # dH: h = 0, so every probability is 2^-16; positive W but for the target's row
    T, V, D = 2560, 65536, 2048
    h = torch.zeros(T, D, device="cuda", dtype=F16)
    w = (0.5 + 0.5 * torch.rand(V, D, device="cuda", generator=gen)).to(F16)
    w[3] = 0
    y = torch.full((T,), 3, device="cuda")
    g = torch.ones(T, device="cuda")
    _, lse = lib.linear_cross_entropy(h, w, y)
    dh, _ = lib.linear_cross_entropy_backward(h, w, y, lse, g, want_weight=False)
    finished()
    assert abs(mean_error(dh[9], w.double().mean(dim=0))) <= bound(D)
