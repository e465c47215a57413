"""The tensor losses in torch's graph of gradients: a loss of tensors that
require a gradient carries it, and what has none says so."""
import math

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
    """The functions on host tensors with the library's calls left out: `calls` lists them."""
    from tiled_dense_gemm_02_gb300 import loss
    calls = []
    monkeypatch.setattr(loss, "_call", lambda torch, device, function, *rest: calls.append(function.__name__))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    return calls


def inputs(device="cpu", T=40, V=300, D=64, K=5, dtype=torch.bfloat16):
    gen = torch.Generator(device=device).manual_seed(0)
    h = torch.randn(T, D, device=device, generator=gen).to(dtype)
    w = (torch.randn(V, D, device=device, generator=gen) * (2.0 / math.sqrt(D))).to(dtype)
    y = torch.randint(0, V, (T,), device=device, generator=gen)
    ids = torch.randint(0, V, (T, K), device=device, generator=gen)
    return h, w, y, ids, torch.randn(T, K, device=device, generator=gen)


def test_the_graph_calls_the_backward_function(tg, on_host):
    h, w, y, ids, logits = inputs()
    w.requires_grad_()
    loss, lse = tg.linear_cross_entropy(h, w, y)
    assert loss.requires_grad
    loss.sum().backward()
    assert on_host == ["tgemm_xent_forward", "tgemm_xent_backward"] and w.grad.shape == w.shape and h.grad is None
    h.requires_grad_()
    loss, lse = tg.linear_distillation(h, w, ids, logits)
    loss.mean().backward()
    assert on_host[2:] == ["tgemm_distill_forward", "tgemm_distill_backward"] and h.grad.shape == h.shape


def test_nothing_is_recorded_where_nothing_is_asked_for(tg, on_host):
    h, w, y, ids, logits = inputs()
    assert not tg.linear_cross_entropy(h, w, y)[0].requires_grad
    w.requires_grad_()
    with torch.no_grad():
        assert not tg.linear_cross_entropy(h, w, y)[0].requires_grad
        assert not tg.linear_distillation(h, w, ids, logits.requires_grad_())[0].requires_grad


def test_what_has_no_gradient_is_refused(tg, on_host):
    h, w, y, ids, logits = inputs()
    w.requires_grad_()
    loss, lse = tg.linear_cross_entropy(h, w, y)
    with pytest.raises(RuntimeError, match="lse"):
        (loss + lse).sum().backward()
    with pytest.raises(ValueError, match="teacher_logits"):
        tg.linear_distillation(h, w, ids, logits.requires_grad_())


def test_inputs_changed_before_the_backward_call_are_noticed(tg, on_host):
    h, w, y, _, _ = inputs()
    w.requires_grad_()
    loss, _ = tg.linear_cross_entropy(h, w, y)
    y.fill_(0)
    with pytest.raises(RuntimeError, match="modified"):
        loss.sum().backward()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("kind", ["xent", "distill"])
def test_gradients_are_those_of_the_backward_functions(tg, kind, T):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h, w, y, ids, logits = inputs("cuda", T=T)
    more = {"label_smoothing": 0.1, "z_loss": 1e-3, "scale": 0.5} if kind == "xent" else {"temperature": 2.0}
    lists = (y,) if kind == "xent" else (ids, logits)
    forward = tg.linear_cross_entropy if kind == "xent" else tg.linear_distillation
    backward = tg.linear_cross_entropy_backward if kind == "xent" else tg.linear_distillation_backward
    g = torch.rand(T, device="cuda")
    loss, lse = forward(h, w, *lists, **more)
    dh, dw = backward(h, w, *lists, lse, g, **more)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side.cuda_stream):
        a, b = h.clone().requires_grad_(), w.clone().requires_grad_()
        torch.cuda.synchronize()
        got, got_lse = forward(a, b, *lists, stream=stream, **more)
        torch.cuda.synchronize()
        (g * got).sum().backward()
        torch.cuda.synchronize()
        assert torch.equal(got, loss) and torch.equal(got_lse, lse)
        assert torch.equal(a.grad, dh) and torch.equal(b.grad, dw)
    # one of the two, and an expanded gradient (that of a sum)
    b = w.clone().requires_grad_()
    forward(h, b, *lists, **more)[0].sum().backward()
    assert torch.equal(b.grad, backward(h, w, *lists, lse, torch.ones(T, device="cuda"), want_hidden=False, **more)[1])
