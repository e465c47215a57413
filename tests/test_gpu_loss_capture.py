"""Steps of the vocabulary-head losses captured in a CUDA graph, one for each way
they take: replayed on new inputs they give the bits of plain calls."""
import math

import pytest
import torch

from tests import gpu_harness as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    H.tg()
    torch.cuda.set_device(0)


def inputs(T, V, D, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.randn(T, D, device="cuda", generator=gen).to(dtype)
    w = (torch.randn(V, D, device="cuda", generator=gen) * (2.0 / math.sqrt(D))).to(dtype)
    y = torch.randint(0, V, (T,), device="cuda", generator=gen)
    y[torch.rand(T, device="cuda", generator=gen) < 0.3] = -100
    ids = torch.randint(0, V, (T, 6), device="cuda", generator=gen)
    return h, w, y, ids, torch.randn(T, 6, device="cuda", generator=gen), torch.rand(T, device="cuda", generator=gen)


@pytest.mark.parametrize("kind", ["xent", "distill"])
@pytest.mark.parametrize("T,V,D,dtype", [(1, 1500, 128, torch.bfloat16), (1, 1500, 131, torch.float16),
                                         (3, 1500, 128, torch.float32), (8, 1500, 129, torch.float32),
                                         (16, 16500, 64, torch.float32), (20, 1500, 64, torch.float32),
                                         (70, 1500, 2100, torch.bfloat16), (300, 1500, 127, torch.float16),
                                         (100, 1500, 600, torch.float32)])
def test_a_captured_step_replays(T, V, D, dtype, kind):
    lib = H.tg()
    held = inputs(T, V, D, dtype, 1)

    def step():
        h, w, y, ids, logits, g = held
        if kind == "xent":
            loss, lse = lib.linear_cross_entropy(h, w, y)
            return (loss, lse) + lib.linear_cross_entropy_backward(h, w, y, lse, g)
        loss, lse = lib.linear_distillation(h, w, ids, logits)
        return (loss, lse) + lib.linear_distillation_backward(h, w, ids, logits, lse, g)

    step()  # first calls set kernel attributes and device records
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (2, 3):
        for x, new in zip(held, inputs(T, V, D, dtype, seed)):
            x.copy_(new)
        graph.replay()
        for x, want in zip(got, step()):
            assert torch.equal(x, want)
    assert lib.device_status(torch.cuda.current_stream().cuda_stream) == lib.OK
