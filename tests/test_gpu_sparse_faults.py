"""Failure detection in the experts' products without a GPU fault: a limit of one microsecond
on the waits of calls whose products take longer."""
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


class Step:
    """Calls through the C ABI on buffers of their own."""

    def __init__(self, T, E, k, D, F, dtype, code):
        lib = H.tg()
        gen = torch.Generator(device="cuda").manual_seed(T + D)

        def normal(*shape):
            return torch.randn(*shape, device="cuda", generator=gen)

        self.sizes, self.code = (T, E, k, D, F), code
        self.x, self.g = normal(T, D).to(dtype), (0.1 * normal(T, D)).to(dtype)
        self.w_in, self.w_out = (normal(E, 2 * F, D) / math.sqrt(D)).to(dtype), (normal(E, D, F) / math.sqrt(F)).to(dtype)
        self.ids, self.weights = torch.topk(normal(T, E), k, dim=1).indices, torch.rand(T, k, device="cuda", generator=gen)
        self.results = [torch.empty_like(v) for v in (self.x, self.x, self.x, self.w_in, self.w_out, self.weights)]
        self.saved = torch.empty(lib.experts_saved_size(*self.sizes, code)[1], dtype=torch.uint8, device="cuda")
        need = [lib.experts_workspace_size(b, *self.sizes, self.w_in.data_ptr(), D, self.w_out.data_ptr(), F, code)[1] for b in (0, 1)]
        self.ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
        self.guard = torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda")
        self.operands = (self.x.data_ptr(), D, self.w_in.data_ptr(), D, self.w_out.data_ptr(), F)

    def end(self, us):
        return H.tg().ExpertsOptions(wait_timeout_us=us), self.ws.data_ptr(), self.ws.numel(), torch.cuda.current_stream().cuda_stream

    def forward(self, us=0, save=False):
        return H.tg().experts_forward(*self.sizes, *self.operands, self.ids.data_ptr(), self.weights.data_ptr(), self.code,
                                      self.results[1 if save else 0].data_ptr(), self.sizes[3], self.saved.data_ptr() if save else 0,
                                      self.saved.numel() if save else 0, *self.end(us))

    def save(self, us=0):
        return self.forward(us, True)

    def backward(self, us=0, wanted=(1, 1, 1, 1)):
        D, F = self.sizes[3:]
        p = [r.data_ptr() if w else 0 for r, w in zip(self.results[2:], wanted)]
        return H.tg().experts_backward(*self.sizes, *self.operands, self.weights.data_ptr(), self.saved.data_ptr(), self.saved.numel(),
                                       self.g.data_ptr(), D, self.code, p[0], D, p[1], D, p[2], F, p[3], *self.end(us))


def status():
    return H.tg().device_status(torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("T,E,k,D,F,dtype,code", [(3000, 3, 2, 2048, 1024, torch.bfloat16, 2), (700, 3, 2, 2048, 1000, torch.bfloat16, 2),
                                                  (3000, 3, 2, 2048, 1024, torch.float16, 1), (700, 3, 2, 2050, 1024, torch.float16, 1)],
                         ids=["bf16", "bf16_gathering", "f16", "f16_odd"])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(T, E, k, D, F, dtype, code):
    lib = H.tg()
    step = Step(T, E, k, D, F, dtype, code)
    for call in (step.forward, step.save, step.backward):
        assert call() == lib.OK
    assert status() == lib.OK
    want = [r.clone() for r in step.results]
    for call in (step.forward, step.save):
        assert call(us=1) == lib.OK
        assert status() == lib.ERR_DEVICE_TIMEOUT
        assert status() == lib.OK
    assert step.save() == lib.OK and status() == lib.OK
    for wanted in ((1, 1, 1, 1), (1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1)):
        assert step.backward(us=1, wanted=wanted) == lib.OK
        assert status() == lib.ERR_DEVICE_TIMEOUT, wanted
        assert status() == lib.OK
    assert bool((step.guard == 7).all())
    for call in (step.forward, step.save, step.backward):
        assert call() == lib.OK
    assert status() == lib.OK
    for got, w in zip(step.results, want):
        assert torch.equal(got, w)
