"""Routing on the GPU against its definition in 64 bits (tests/route_reference.py):
sizes, ties, masks, groups and types where it can go wrong."""
import itertools
import math

import pytest
import torch

from tests import gpu_harness as H
from tests.route_reference import Routed

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAMES = {BF16: "bf16", F16: "f16", F32: "f32"}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    H.tg()
    torch.cuda.set_device(0)


def rows(T, E, dtype, seed=0, pad=0, spread=1.5):
    gen = torch.Generator(device="cuda").manual_seed(100 + seed)
    return (spread * torch.randn(T, E + pad, device="cuda", generator=gen)).to(dtype)[:, :E], gen


def both(logits, k, gen, bias=None, **more):
    lib = H.tg()
    ids, weights = lib.route_experts(logits, k, bias=bias, **more)
    want = Routed(logits, k, bias=bias, **more)
    want.check(ids, weights)
    g = torch.randn(weights.shape, device="cuda", generator=gen)
    options = {n: more[n] for n in ("scoring", "renormalize", "scale") if n in more}
    want.check_gradient(lib.route_experts_backward(logits, ids, g, **options), g)
    return ids, weights


SIZES = [(1, 1, 1), (1, 8, 8), (3, 31, 2), (5, 32, 32), (17, 33, 4), (64, 60, 4), (129, 64, 6), (33, 128, 8),
         (257, 200, 10), (100, 256, 8), (40, 257, 16), (30, 512, 3), (21, 1000, 32), (9, 1024, 1)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=NAMES.get)
def test_every_kind_of_scores(T, E, k, dtype):
    for i, (scoring, biased, renormalize) in enumerate(itertools.product(("softmax", "sigmoid"), (False, True), (False, True))):
        logits, gen = rows(T, E, dtype, seed=i, pad=i % 3)
        bias = 0.2 * torch.randn(E, device="cuda", generator=gen) if biased else None
        both(logits, k, gen, bias, scoring=scoring, renormalize=renormalize, scale=(1.0, 2.5)[i % 2])


@pytest.mark.parametrize("E,groups,top_groups,k", [(8, 8, 3, 3), (32, 4, 1, 8), (60, 6, 2, 5), (256, 8, 4, 8), (64, 32, 7, 6),
                                                   (100, 10, 10, 12), (1024, 32, 5, 32), (96, 3, 2, 1)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_groups(E, groups, top_groups, k, group_score):
    for i, (scoring, biased) in enumerate(itertools.product(("softmax", "sigmoid"), (False, True))):
        logits, gen = rows(203, E, (F32, BF16)[i % 2], seed=i)
        bias = 0.2 * torch.randn(E, device="cuda", generator=gen) if biased else None
        both(logits, k, gen, bias, scoring=scoring, groups=groups, top_groups=top_groups, group_score=group_score)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_masks_down_to_rows_with_nothing_left(scoring, groups):
    for dtype, biased in itertools.product((BF16, F32), (False, True)):
        logits, gen = rows(300, 48, dtype, seed=5)
        logits = logits.clone()
        gone = torch.rand(300, 48, device="cuda", generator=gen) < torch.linspace(0, 1.05, 300, device="cuda")[:, None]
        logits[gone] = -math.inf
        logits[7] = torch.finfo(dtype).min  # the type's lowest number is a number
        bias = 0.1 * torch.randn(48, device="cuda", generator=gen) if biased else None
        ids, weights = both(logits, 6, gen, bias, scoring=scoring, groups=groups, top_groups=max(1, groups // 2),
                            group_score="top2")
        assert bool((ids[-1] == -1).all()) and bool((weights[-1] == 0).all()) and not bool((ids[7] == -1).any())
        picked = torch.gather(gone, 1, ids.clamp_min(0))
        assert not bool((picked & (ids >= 0)).any())


def test_a_bias_of_minus_infinity_masks_too():
    logits, gen = rows(50, 16, F32)
    bias = torch.zeros(16, device="cuda")
    bias[3:] = -math.inf
    ids, weights = H.tg().route_experts(logits, 5, bias=bias)
    assert bool((ids[:, 3:] == -1).all()) and bool((weights[:, 3:] == 0).all())
    assert torch.equal(ids[:, :3].sort(dim=1).values, torch.arange(3, device="cuda").expand(50, 3))


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=NAMES.get)
def test_ties_go_to_the_lowest_index(dtype):
    gen = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randint(-2, 3, (400, 150), device="cuda", generator=gen).to(dtype)
    logits[0] = 0.0
    logits[1, ::2] = -0.0
    logits[1, 1::2] = 0.0
    for bias in (None, torch.zeros(150, device="cuda")):
        for scoring in ("softmax", "sigmoid"):
            ids, _ = both(logits, 8, gen, bias, scoring=scoring)
            assert ids[0].tolist() == ids[1].tolist() == list(range(8))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,group_score", [(1, "max"), (8, "max"), (8, "top2")])
def test_keys_closer_than_fp32_resolves(scoring, groups, group_score):
    """A bias that cancels the scores up to fp32's last bits: what is left decides, and only 64 bits see it."""
    E = 64
    logits, gen = rows(1, E, F32, seed=9)
    score = Routed(logits, 1, scoring=scoring).score[0]
    bias = (0.5 - score).float()
    logits = logits.expand(40, E).contiguous()
    logits[20:] += 1e-6 * torch.randn(20, E, device="cuda", generator=gen)
    both(logits, 8, gen, bias, scoring=scoring, groups=groups, top_groups=max(1, groups // 2), group_score=group_score)


def test_far_logits():
    """Sigmoids that underflow share their weight as the real numbers do; softmax over thousands."""
    logits = torch.tensor([[-200.0, -201.0, -202.0, -300.0], [-90.0, -95.0, -100.0, 5.0], [80.0, 90.0, 30.0, 100.0],
                           [1e4, 1e4 - 1, -1e4, 0.0], [-3e38, 3e38, 0.0, 1.0]], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    for scoring in ("softmax", "sigmoid"):
        both(logits, 2, gen, scoring=scoring)
    _, w = H.tg().route_experts(logits, 3, scoring="sigmoid")
    want = torch.softmax(torch.tensor([-200.0, -201.0, -202.0], dtype=torch.float64), 0)
    assert torch.allclose(w[0].double().cpu(), want, rtol=3e-7)


def test_nan_ranks_first_and_stays():
    logits, _ = rows(6, 40, F32)
    logits[2, 17] = math.nan
    logits[4] = -math.inf
    logits[4, 9] = math.nan
    clean = [0, 1, 3, 5]
    for scoring in ("softmax", "sigmoid"):
        ids, w = H.tg().route_experts(logits, 4, scoring=scoring)
        assert int(ids[2, 0]) == 17 and bool(w[2].isnan().all()) and int(ids[4, 0]) == 9 and int(ids[4, 1]) == -1
        want = Routed(logits[clean], 4, scoring=scoring)
        want.check(ids[clean], w[clean])
    ids, w = H.tg().route_experts(logits, 4, scoring="sigmoid", renormalize=False)
    assert bool(w[2, 0].isnan()) and not bool(w[2, 1:].isnan().any())


def test_rows_of_a_long_batch_with_a_wide_pitch():
    """Rows past 2^31 elements from the first."""
    T, E, ld = 70_000, 16, 40_000
    wide = torch.empty(T, ld, dtype=BF16, device="cuda")
    logits, gen = rows(T, E, BF16, seed=3)
    wide[:, :E] = logits
    both(wide[:, :E], 2, gen)


def test_empty_batch():
    lib = H.tg()
    ids, w = lib.route_experts(torch.empty(0, 8, device="cuda"), 2)
    assert ids.shape == w.shape == (0, 2)
    assert lib.route_experts_backward(torch.empty(0, 8, device="cuda"), ids, w).shape == (0, 8)


def test_backward_leaves_out_unused_and_bad_places_and_adds_repeats():
    lib = H.tg()
    logits, gen = rows(3, 20, F32)
    ids = torch.tensor([[4, -1, 7], [30, 5, -1], [6, 6, -7]], device="cuda")
    g = torch.randn(3, 3, device="cuda", generator=gen)
    g[0, 1] = math.nan
    d = lib.route_experts_backward(logits, ids, g, scoring="sigmoid", renormalize=False)
    s = torch.sigmoid(logits.double())
    want = torch.zeros(3, 20, dtype=torch.float64, device="cuda")
    for r, e, j in ((0, 4, 0), (0, 7, 2), (1, 5, 1), (2, 6, 0), (2, 6, 1)):
        want[r, e] += g[r, j].double() * s[r, e] * (1 - s[r, e])
    assert torch.allclose(d.double(), want, rtol=1e-6, atol=1e-12)


def test_gradient_through_torch_and_differences():
    lib = H.tg()
    logits, gen = rows(50, 24, F32, seed=4)
    g = torch.randn(50, 4, device="cuda", generator=gen)
    for scoring, renormalize in itertools.product(("softmax", "sigmoid"), (False, True)):
        more = {"scoring": scoring, "renormalize": renormalize, "scale": 1.5}
        x = logits.clone().requires_grad_()
        ids, w = lib.route_experts(x, 4, **more)
        assert w.requires_grad and not ids.requires_grad
        (g * w).sum().backward()
        assert torch.equal(x.grad, lib.route_experts_backward(logits, ids, g, **more))
        # central differences of the definition, picks held: h^2 and 2^-53 / h leave 1e-9
        h, shift = 1e-4, torch.randn(50, 24, dtype=torch.float64, device="cuda", generator=gen)

        def loss(v):
            v = v.double()
            p = torch.softmax(v, 1) if scoring == "softmax" else torch.sigmoid(v)
            p = p.gather(1, ids)
            return 1.5 * (g.double() * (p / p.sum(1, keepdim=True) if renormalize else p)).sum()

        slope = (loss(logits.double() + h * shift) - loss(logits.double() - h * shift)) / (2 * h)
        got = (x.grad.double() * shift).sum()
        size = (x.grad.double() * shift).abs().sum()
        assert abs(float(got - slope)) <= 2.0 ** -19 * float(size) + 1e-6


def test_calls_are_captured_and_follow_their_stream():
    lib = H.tg()
    logits, gen = rows(300, 128, BF16)
    g = torch.randn(300, 8, device="cuda", generator=gen)
    bias = 0.1 * torch.randn(128, device="cuda", generator=gen)

    def step():
        ids, w = lib.route_experts(logits, 8, bias=bias)
        return ids, w, lib.route_experts_backward(logits, ids, g)

    want = step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ids, w = lib.route_experts(logits, 8, bias=bias, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(ids, want[0]) and torch.equal(w, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (7, 8):
        logits.copy_(rows(300, 128, BF16, seed=seed)[0])
        graph.replay()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
