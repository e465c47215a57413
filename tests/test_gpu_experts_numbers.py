"""Numbers at the ends of their range in the experts' products: where a computation that is right in the
middle of it overflows, underflows or loses what lies beside a larger number (tests/experts_numbers.py)."""
import math

import pytest
import torch

from tests import gpu_harness as H
from tests.experts_numbers import Numbers

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
NAMES = {BF16: "bf16", F16: "f16"}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    H.tg()
    torch.cuda.set_device(0)


def normals(seed):
    gen = torch.Generator(device="cuda").manual_seed(9000 + seed)
    return lambda *shape: torch.randn(*shape, device="cuda", generator=gen)


def layer(T, E, k, D, F, dtype, seed=0):
    normal = normals(seed)
    x, w_in, w_out = normal(T, D), normal(E, 2 * F, D) / math.sqrt(D), normal(E, D, F) / math.sqrt(F)
    ids = torch.topk(normal(T, E), k, dim=1).indices
    return x.to(dtype), w_in.to(dtype), w_out.to(dtype), ids, torch.rand_like(ids.float()), (0.1 * normal(T, D)).to(dtype), normal


def gradients(x, w_in, w_out, ids, weights, g, **more):
    lib = H.tg()
    out, saved = lib.expert_mlp(x, w_in, w_out, ids, weights, save=True)
    got = dict(zip(("dx", "dw_in", "dw_out", "dw"), lib.expert_mlp_backward(x, w_in, w_out, ids, weights, saved, g, **more)))
    assert lib.device_status(torch.cuda.current_stream().cuda_stream) == lib.OK
    return {"out": out, **{n: v for n, v in got.items() if v is not None}}


def check(*args):
    got = gradients(*args)
    Numbers(*args).check(**got)
    return got


@pytest.mark.parametrize("T,F", [(70, 64), (300, 63)])
def test_fp16_gradients_that_grow_with_the_depth(T, F):
    """dg and du sum over D: with a constant gradient and weights of one sign they are thousands of times the gradient."""
    D, E = 4096, 2
    x, w_in, w_out, ids, _, _, normal = layer(T, E, 1, D, F, F16, seed=F)
    g = torch.full((T, D), 2.0 ** -10, device="cuda").half()
    check(4 * x, w_in, w_out.abs(), ids, torch.ones(T, 1, device="cuda"), g)


def test_fp16_gradients_of_large_inputs():
    """u of size 60: du is, and dg is 60 times as large."""
    x, w_in, w_out, ids, _, g, _ = layer(90, 2, 1, 8192, 64, F16)
    check((60 * x.float()).half(), w_in, w_out / 64, ids, torch.ones(90, 1, device="cuda"), g / 64)


def test_fp16_gradients_of_large_weights():
    x, w_in, w_out, ids, _, g, _ = layer(256, 4, 1, 512, 1024, F16)
    check(x, w_in, (2000 * w_out.float()).half(), ids, torch.ones(256, 1, device="cuda"), g / 2)


@pytest.mark.parametrize("size", [2.0 ** -20, 2.0 ** -12, 1.0, 2.0 ** 8])
@pytest.mark.parametrize("odd", [0, 1])
def test_fp16_gradients_whatever_the_output_weights_are(size, odd):
    """dg and du over the gradient from 2^-20 to 2^8; the operands stay in the middle of fp16's range."""
    x, w_in, w_out, ids, weights, g, _ = layer(200, 3, 2, 256, 128 - odd, F16, seed=3)
    a, b = (2.0 ** 8, size / 2 ** 8) if size >= 1 else (2.0 ** -8, size * 2 ** 8)
    # a part of the factor in W_out, the rest in x's gates and ups
    check((x.float() * math.sqrt(max(1.0, b))).half(), w_in, (w_out.float() * a * min(1.0, b)).half(), ids, weights, (g.float() / 64).half())


@pytest.mark.parametrize("w", [1e-2, 1e-5, 1e-6, 1e-9])
def test_fp16_places_of_small_weight_keep_their_gradients(w):
    """w h below fp16's numbers: dW_out, with gradients of size 64, is well within them."""
    x, w_in, w_out, ids, _, g, _ = layer(300, 3, 2, 128, 96, F16)
    got = check((3 * x.float()).half(), w_in, w_out, ids, torch.full((300, 2), w, device="cuda"), (640 * g.float()).half())
    want = Numbers((3 * x.float()).half(), w_in, w_out, ids, torch.full((300, 2), w, device="cuda"), (640 * g.float()).half())
    if w >= 1e-6:  # in the norm: w h's rounding and the last one, each below half a step
        off = (got["dw_out"].double() - want.dw_out).norm() / want.dw_out.norm()
        assert float(off) <= 2.0 ** -11, float(off)


def test_fp16_rows_and_experts_of_very_different_weight():
    """Rows and experts whose gradients lie 2^-20 apart: each row's dx and each expert's dW keep their bits."""
    x, w_in, w_out, ids, _, g, normal = layer(400, 4, 1, 128, 96, F16)
    ids = torch.arange(400, device="cuda")[:, None] % 4
    weights = torch.ones(400, 1, device="cuda")
    weights[ids == 1] = 2.0 ** -20
    weights[ids == 2] = 2.0 ** -30
    weights[ids == 3] = 2.0 ** -20
    weights[3:100:4] = 1.0  # expert 3: both kinds
    g = (640 * g.float()).half()
    got = check(x, w_in, w_out, ids, weights, g)
    want = Numbers(x, w_in, w_out, ids, weights, g)
    large = want.dx.abs().amax(dim=1) >= 2.0 ** -12  # rows whose dx fp16 holds with all bits
    off = (got["dx"].double() - want.dx).norm(dim=1) / want.dx.norm(dim=1)
    assert int(large.sum()) > 100 and float(off[large].max()) <= 2.0 ** -10


def test_fp16_rows_beside_an_infinite_gradient():
    """A row whose gradient is infinite takes nothing from the other rows and the other experts."""
    x, w_in, w_out, ids, weights, g, _ = layer(130, 4, 1, 128, 96, F16)
    g[7, 5] = math.inf
    g[9, 0] = math.nan
    bad = torch.zeros(130, dtype=torch.bool, device="cuda")
    bad[[7, 9]] = True
    got = gradients(x, w_in, w_out, ids, weights, g)
    hit = torch.unique(ids[bad])
    keep = torch.tensor([e for e in range(4) if e not in hit.tolist()], device="cuda")
    assert keep.numel() > 0
    want = Numbers(x, w_in, w_out, ids, weights, torch.where(bad[:, None], torch.zeros_like(g), g))
    want.check(rows=~bad, experts=keep, **got)
    assert not bool(got["dx"][bad].isfinite().any())


@pytest.mark.parametrize("dtype", [BF16, F16], ids=NAMES.get)
@pytest.mark.parametrize("D,F", [(600, 70), (1100, 300)])
def test_gradients_do_not_depend_on_which_are_asked_for(D, F, dtype):
    """Freezing a router, or some weights, leaves the other gradients' bits: sums of several chunks."""
    x, w_in, w_out, ids, weights, g, _ = layer(300, 4, 2, D, F, dtype, seed=D)
    names = ("dx", "dw_in", "dw_out", "dw")
    want = gradients(x, w_in, w_out, ids, weights, g)
    for mask in range(1, 15):
        wants = dict(zip(("want_hidden", "want_in", "want_out", "want_weights"), [bool(mask >> i & 1) for i in range(4)]))
        got = gradients(x, w_in, w_out, ids, weights, g, **wants)
        assert set(got) == {"out"} | {n for i, n in enumerate(names) if mask >> i & 1}
        for name, v in got.items():
            assert torch.equal(v, want[name]), (mask, name)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=NAMES.get)
@pytest.mark.parametrize("F", [1, 40, 300])
def test_an_infinite_gradient_gives_an_infinite_weight_gradient(F, dtype):
    """Positive numbers all: d_weights is +inf where one gradient is, at widths that do not fill the tiles."""
    x, w_in, w_out, ids, weights, g, _ = layer(50, 2, 1, 64, F, dtype)
    g = g.abs()
    g[3, 5] = math.inf
    got = gradients(x.abs(), w_in.abs(), w_out.abs(), ids, weights, g)
    assert float(got["dw"][3, 0]) == math.inf
    assert bool(got["dw"][torch.arange(50, device="cuda") != 3].isfinite().all())


@pytest.mark.parametrize("T", [40, 300])
def test_bf16_neighbours_of_very_different_size(T):
    """Elements of out and dx far below their neighbours in a row, which bf16 holds: they keep their own bits."""
    E, D, F = 3, 200, 96
    x, w_in, w_out, ids, weights, g, normal = layer(T, E, 2, D, F, BF16, seed=T)
    sizes = torch.tensor([0.0, 0.0, -12.0, -26.0, -29.0, -33.0, -41.0, -45.0, -80.0, 20.0], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(T)
    scale = torch.exp2(sizes[torch.randint(0, 10, (D,), device="cuda", generator=gen)])
    scale[32:64] = 1.0
    scale[33] = 0.0
    w_out = (w_out.float() * scale[:, None]).bfloat16()
    w_in = (w_in.float() * scale.clamp_max(1.0)).bfloat16()
    got = check(x, w_in, w_out, ids, weights, g)
    assert bool((got["out"][:, 33] == 0).all())
    want = Numbers(x, w_in, w_out, ids, weights, g)
    for name in ("out", "dx"):  # the bounds tell them from 0: half of the elements are above twice theirs
        assert float(((getattr(want, name).abs() > 2 * getattr(want, "e_" + name)).float().mean(dim=0) >= 0.5).float().mean()) > 0.9
    plain = H.tg().expert_mlp(x, w_in, w_out, ids, weights)[0]
    Numbers(x, w_in, w_out, ids, weights, g, train=False).check(out=plain)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=NAMES.get)
@pytest.mark.parametrize("T,D,F", [(40, 40_000, 24), (40, 64, 40_000), (30_000, 64, 24)])
def test_long_axes_of_one_sign_stay_within_their_bounds(T, D, F, dtype):
    """Sums of many chunks: a truncation a step and a rounding a chunk, whichever axis is long."""
    x, w_in, w_out, ids, weights, g, _ = layer(T, 2, 1, D, F, dtype, seed=F)
    ids.fill_(1)
    args = (x.abs() / 16 if D > 10_000 else x.abs() / 2, w_in.abs(), w_out.abs() / 4, ids, weights, g.abs() / 64)
    check(*args)
    out = H.tg().expert_mlp(*args[:5])[0]
    Numbers(*args, train=False).check(out=out)


@pytest.mark.parametrize("byte", [0x00, 0x7F, 0xFF])
@pytest.mark.parametrize("T,D,F", [(1, 8, 1), (130, 200, 121), (700, 264, 72)])
def test_fp16_workspaces_hold_anything(T, D, F, byte):
    """Lent to one call after the other, on two streams: each has its own largest numbers."""
    lib = H.tg()
    calls = [layer(T, 5, 2, D, F, F16, seed=s)[:6] for s in (1, 2)]
    calls[1][5].mul_(64)
    want = [gradients(*c) for c in calls]
    n = lib.experts_workspace_size(1, T, 5, 2, D, F, calls[0][1].data_ptr(), D, calls[0][2].data_ptr(), F, lib.F16)[1]
    ws = [torch.full((n,), byte, dtype=torch.uint8, device="cuda") for _ in calls]
    saved = [lib.expert_mlp(*c[:5], save=True)[1] for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for turn in range(2):
        got = [lib.expert_mlp_backward(*calls[i ^ turn][:5], saved[i ^ turn], calls[i ^ turn][5], workspace=ws[i], stream=streams[i].cuda_stream)
               for i in range(2)]
        torch.cuda.synchronize()
        for i in range(2):
            for name, v in zip(("dx", "dw_in", "dw_out", "dw"), got[i]):
                assert torch.equal(v, want[i ^ turn][name]), (turn, name)
