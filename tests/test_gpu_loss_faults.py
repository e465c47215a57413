"""Failure detection in the vocabulary-head losses without a GPU fault: a limit
of one microsecond on the waits of a call whose products take longer."""
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
    """A forward and a backward call through the C ABI on buffers of their own."""

    def __init__(self, T, V, D, dtype, code):
        lib = H.tg()
        gen = torch.Generator(device="cuda").manual_seed(T + D)
        self.sizes, self.code = (T, V, D), code
        self.h = torch.randn(T, D, device="cuda", generator=gen).to(dtype)
        self.w = (torch.randn(V, D, device="cuda", generator=gen) * D ** -0.5).to(dtype)
        self.y = torch.randint(0, V, (T,), device="cuda", generator=gen)
        self.g = torch.rand(T, device="cuda", generator=gen)
        self.loss, self.lse, self.dh, self.dw = (torch.empty(n, device="cuda", dtype=t) for n, t in (
            ((T,), torch.float32), ((T,), torch.float32), ((T, D), dtype), ((V, D), dtype)))
        need = [lib.loss_workspace_size(b, T, V, D, 0, self.w.data_ptr(), D, code)[1] for b in (False, True)]
        self.ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
        self.guard = torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda")

    def options(self, us):
        return H.tg().LossOptions(ignore_index=-100, wait_timeout_us=us)

    def forward(self, us=0):
        T, V, D = self.sizes
        return H.tg().xent_forward(T, V, D, self.h.data_ptr(), D, self.w.data_ptr(), D, self.y.data_ptr(), self.code,
                                   self.loss.data_ptr(), self.lse.data_ptr(), self.options(us), self.ws.data_ptr(),
                                   self.ws.numel(), torch.cuda.current_stream().cuda_stream)

    def backward(self, us=0):
        T, V, D = self.sizes
        return H.tg().xent_backward(T, V, D, self.h.data_ptr(), D, self.w.data_ptr(), D, self.y.data_ptr(),
                                    self.lse.data_ptr(), self.g.data_ptr(), self.code, self.dh.data_ptr(), D,
                                    self.dw.data_ptr(), D, self.options(us), self.ws.data_ptr(), self.ws.numel(),
                                    torch.cuda.current_stream().cuda_stream)


def status():
    return H.tg().device_status(torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("T,V,D,dtype,code", [(600, 20000, 2048, torch.bfloat16, 2), (300, 9000, 1024, torch.float16, 1),
                                              (300, 9000, 1024, torch.float32, 0)], ids=["bf16", "f16", "f32"])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(T, V, D, dtype, code):
    lib = H.tg()
    step = Step(T, V, D, dtype, code)
    assert step.forward() == lib.OK and step.backward() == lib.OK and status() == lib.OK
    want = [x.clone() for x in (step.loss, step.lse, step.dh, step.dw)]
    for call in (step.forward, step.backward):
        assert call(us=1) == lib.OK
        assert status() == lib.ERR_DEVICE_TIMEOUT
        assert status() == lib.OK
    assert bool((step.guard == 7).all())
    assert step.forward() == lib.OK and step.backward() == lib.OK and status() == lib.OK
    for x, y in zip((step.loss, step.lse, step.dh, step.dw), want):
        assert torch.equal(x, y)
