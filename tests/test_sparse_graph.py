"""The tensor functions of a sparse layer and torch's graphs, on the host: what a backward pass reads, what forward
mode is told, and what is written in place.  No call here reaches the GPU."""
import pytest
import torch


@pytest.fixture(scope="module")
def tg():
    from tests.conftest import build_library
    build_library()
    import tiled_dense_gemm_02_gb300 as tg
    return tg


@pytest.fixture
def on_host(tg, monkeypatch):
    """The functions on host tensors with the library's calls left out: `calls` lists their arguments."""
    from tiled_dense_gemm_02_gb300 import experts, grads, loss
    calls = []

    def guarded(torch, device, function, args):
        calls.append((function.__name__, args))
        return tg.OK

    for module in (experts, grads, loss):
        monkeypatch.setattr(module, "_guarded", guarded)
        monkeypatch.setattr(module, "_current_stream", lambda torch, device: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    return calls


def route_options(args):
    from tiled_dense_gemm_02_gb300 import RouteOptions
    return next(a._obj for a in args if hasattr(a, "_obj") and isinstance(a._obj, RouteOptions))


def test_routing_options_that_change_before_the_backward_pass(tg, on_host):
    """A scale or a flag held in a tensor: the gradient is that of the weights that were given."""
    logits = torch.randn(4, 8).requires_grad_()
    scale, renormalize = torch.tensor(2.0), torch.tensor(False)
    _, weights = tg.route_experts(logits, 2, scoring="sigmoid", scale=scale, renormalize=renormalize)
    scale.fill_(3.0)
    renormalize.fill_(True)
    weights.sum().backward()
    (first, forward), (then, backward) = on_host
    assert (first, then) == ("tgemm_route_forward", "tgemm_route_backward")
    for o in (route_options(forward), route_options(backward)):
        assert (o.scoring, o.scale, o.renormalize) == (1, 2.0, 0)


def operands(T=4, E=3, k=2, D=8, F=16):
    return (torch.randn(T, D).bfloat16(), torch.randn(E, 2 * F, D).bfloat16(), torch.randn(E, D, F).bfloat16(),
            torch.zeros(T, k, dtype=torch.int64), torch.rand(T, k))


def test_tangents_of_forward_mode_are_refused(tg, on_host):
    """There is no forward-mode gradient: a dual tensor must not lose its tangent without a word."""
    from torch.autograd import forward_ad
    args = operands()
    logits, bias = torch.randn(4, 8), torch.randn(8)
    y, lists = torch.zeros(4, dtype=torch.int64), (torch.zeros(4, 2, dtype=torch.int64), torch.randn(4, 2))
    weight = torch.randn(10, 8).bfloat16()
    with forward_ad.dual_level():
        def dual(t):
            return forward_ad.make_dual(t, torch.ones_like(t))

        for i in (0, 1, 2, 4):
            with pytest.raises(RuntimeError, match="forward"):
                tg.expert_mlp(*[dual(a) if j == i else a for j, a in enumerate(args)])
        for call in (lambda: tg.route_experts(dual(logits), 2), lambda: tg.route_experts(logits, 2, bias=dual(bias)),
                     lambda: tg.linear_cross_entropy(dual(args[0]), weight, y), lambda: tg.linear_cross_entropy(args[0], dual(weight), y),
                     lambda: tg.linear_distillation(dual(args[0]), weight, *lists), lambda: tg.linear_distillation(args[0], dual(weight), *lists),
                     lambda: tg.linear_distillation(args[0], weight, lists[0], dual(lists[1]))):
            with pytest.raises(RuntimeError, match="forward"):
                call()
        assert on_host == []
        tg.expert_mlp(*args)  # tensors without a tangent
        tg.route_experts(logits, 2, bias=bias)
        tg.linear_cross_entropy(args[0], weight, y)
    assert len(on_host) == 3


def test_what_is_clipped_in_place_is_seen_as_changed(tg, on_host):
    """torch's graph notices that a tensor which it keeps was written."""
    a, b, c = torch.randn(5), torch.randn(7).half(), torch.randn(3)
    before = [t._version for t in (a, b, c)]
    tg.gradient_norm([a, b])
    assert [t._version for t in (a, b, c)] == before
    tg.clip_gradients([a, b], 1.0)
    assert a._version > before[0] and b._version > before[1]
    seen = a._version
    tg.clip_gradients([a], 1.0, outputs=[torch.empty(5)])
    assert a._version == seen
    out = torch.empty(5)
    seen = out._version
    tg.clip_gradients([a], 1.0, outputs=[out])
    assert out._version > seen
    with torch.inference_mode():
        kept = torch.randn(4)
    tg.clip_gradients([kept, c], 1.0)  # has no counter
    assert c._version > before[2]
    x = torch.randn(5, requires_grad=True)
    y = (x * a).sum()
    tg.clip_gradients([a], 1.0)
    with pytest.raises(RuntimeError, match="modified"):
        y.backward()
