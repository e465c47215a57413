"""The experts' products on the GPU against their definition in 64 bits
(tests/experts_reference.py), at the sizes, lists and layouts where they can go
wrong, through the tensor functions and through the C ABI."""
import math

import pytest
import torch

from tests import gpu_harness as H
from tests.experts_reference import Experts

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
NAMES = {BF16: "bf16", F16: "f16"}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    H.tg()
    torch.cuda.set_device(0)


def layer(T, E, k, D, F, dtype, seed=0, pad=0, skew=0.5):
    gen = torch.Generator(device="cuda").manual_seed(2000 + seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    x = normal(T, D + pad).to(dtype)[:, :D]
    w_in = (normal(E, 2 * F, D) / math.sqrt(D)).to(dtype)
    w_out = (normal(E, D, F) / math.sqrt(F)).to(dtype)
    ids = torch.topk(normal(T, E) + skew * normal(E), k, dim=1).indices
    weights = torch.rand(T, k, device="cuda", generator=gen)
    return x, w_in, w_out, ids, weights, (0.1 * normal(T, D)).to(dtype), gen


def finished():
    lib = H.tg()
    assert lib.device_status(torch.cuda.current_stream().cuda_stream) == lib.OK
    return lib


def both(x, w_in, w_out, ids, weights, g, **more):
    lib = H.tg()
    plain, none = lib.expert_mlp(x, w_in, w_out, ids, weights)
    assert none is None
    out, saved = lib.expert_mlp(x, w_in, w_out, ids, weights, save=True)
    dx, dw_in, dw_out, dw = lib.expert_mlp_backward(x, w_in, w_out, ids, weights, saved, g, **more)
    finished()
    return plain, {"out": out, "dx": dx, "dw_in": dw_in, "dw_out": dw_out, "dw": dw}


def check(x, w_in, w_out, ids, weights, g):
    plain, got = both(x, w_in, w_out, ids, weights, g)
    Experts(x, w_in, w_out, ids, weights, g).check(**got)
    Experts(x, w_in, w_out, ids, weights).check(out=plain)
    return got


SHAPES = [(1, 1, 1, 8, 8), (1, 4, 2, 64, 64), (2, 3, 3, 1, 1), (3, 5, 2, 72, 40), (7, 2, 1, 65, 33), (17, 8, 4, 128, 256),
          (33, 4, 2, 200, 136), (64, 16, 8, 256, 128), (100, 3, 2, 130, 250), (129, 2, 2, 512, 64), (256, 8, 2, 192, 384),
          (257, 1, 1, 264, 72), (300, 6, 3, 520, 520), (513, 4, 2, 100, 700), (700, 2, 1, 640, 272), (1000, 10, 3, 331, 170),
          (31, 200, 5, 64, 24)]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=NAMES.get)
@pytest.mark.parametrize("T,E,k,D,F", SHAPES)
def test_forward_and_backward_match_the_definition(T, E, k, D, F, dtype):
    check(*layer(T, E, k, D, F, dtype, seed=T + D)[:6])


@pytest.mark.parametrize("T,E,k", [(1, 64, 8), (2, 5, 3), (4, 8, 8), (32, 2, 1), (33, 2, 1)])
@pytest.mark.parametrize("D,F", [(256, 128), (264, 72), (200, 33), (2048, 1000)])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=NAMES.get)
def test_a_few_places(T, E, k, D, F, dtype):
    """Both ways of a short forward call: weights read place by place, and the tensor cores (the step's forward)."""
    x, w_in, w_out, ids, weights, g, _ = layer(T, E, k, D, F, dtype, seed=T)
    ids[0, 0] = -1
    if T > 1:
        ids[1] = -5
    check(x, w_in, w_out, ids, weights, g)


@pytest.mark.parametrize("T,E,k", [(400, 3, 2), (1025, 2, 2), (3000, 40, 4), (20000, 9, 8), (150_000, 5, 1)])
def test_sorts_of_every_size(T, E, k):
    """One block's sort, many blocks' of 512 places, and of 2048; popular and empty experts."""
    x, w_in, w_out, ids, weights, g, gen = layer(T, E, k, 64, 32, BF16, seed=E, skew=3.0)
    ids[torch.rand(T, k, device="cuda", generator=gen) < 0.2] = -1
    ids[ids == 1] = 0
    got = check(x, w_in, w_out, ids, weights, g)
    assert bool((got["dw_in"][1] == 0).all()) and bool((got["dw_out"][1] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F16], ids=NAMES.get)
@pytest.mark.parametrize("T", [3, 60, 700])
def test_unused_places_whatever_the_rows_hold(T, dtype):
    """Rows without a used place, NaN and infinities in them: zeros, and no other row or gradient sees them."""
    x, w_in, w_out, ids, weights, g, gen = layer(T, 6, 3, 136, 80, dtype, seed=T)
    dead = torch.rand(T, device="cuda", generator=gen) < 0.4
    dead[1] = True
    ids[dead] = -1
    ids[::2, 1] = -9
    clean = x.clone()
    x[dead] = float("nan")
    x[1] = float("inf")
    g = g.clone()
    g[dead] = float("nan")
    weights[dead] = float("nan")
    weights[ids < 0] = float("inf")
    plain, got = both(x, w_in, w_out, ids, weights, g)
    want = Experts(clean, w_in, w_out, ids, weights, torch.where(dead[:, None], torch.zeros_like(g), g))
    want.check(**got)
    for name in ("out", "dx", "dw"):
        assert bool((got[name][dead] == 0).all()), name
    assert bool((plain[dead] == 0).all()) and bool((got["dw"][ids < 0] == 0).all())


@pytest.mark.parametrize("T", [1, 40, 900])
def test_ids_past_the_experts_are_seen_in_their_rows_alone(T):
    x, w_in, w_out, ids, weights, g, _ = layer(T, 4, 2, 64, 48, BF16)
    ids[0, 1] = 4
    ids[T // 2, 0] = 1 << 40
    bad = (ids >= 4).any(dim=1)
    plain, got = both(x, w_in, w_out, ids, weights, g)
    used = torch.where(ids >= 4, torch.full_like(ids, -1), ids)
    want = Experts(x, w_in, w_out, used, weights, g)
    assert bool(plain[bad].isnan().all()) and bool(got["out"][bad].isnan().all()) and bool(got["dx"][bad].isnan().all())
    assert bool(got["dw"][ids >= 4].isnan().all()) and not bool(got["dw"][ids < 4].isnan().any())
    want.check(dw_in=got["dw_in"], dw_out=got["dw_out"])
    for name in ("out", "dx"):
        assert bool(((got[name].double() - getattr(want, name)).abs() <= getattr(want, "e_" + name))[~bad].all())


def test_an_expert_listed_twice_counts_twice():
    x, w_in, w_out, ids, weights, g, _ = layer(50, 3, 3, 64, 64, BF16)
    ids[:, 1] = ids[:, 0]
    ids[7] = 2
    check(x, w_in, w_out, ids, weights, g)


@pytest.mark.parametrize("T", [40, 600])
def test_nothing_used_at_all(T):
    x, w_in, w_out, ids, weights, g, _ = layer(T, 3, 2, 64, 64, F16)
    ids.fill_(-1)
    plain, got = both(x, w_in, w_out, ids, weights, g)
    for v in [plain, *got.values()]:
        assert bool((v == 0).all())


def test_no_rows():
    lib = H.tg()
    x, w_in, w_out, ids, weights, g, _ = layer(2, 3, 2, 64, 32, BF16)
    out, saved = lib.expert_mlp(x[:0], w_in, w_out, ids[:0], weights[:0], save=True)
    dx, dw_in, dw_out, dw = lib.expert_mlp_backward(x[:0], w_in, w_out, ids[:0], weights[:0], saved, g[:0])
    finished()
    assert out.shape == dx.shape == (0, 64) and dw.shape == (0, 2)
    assert bool((dw_in == 0).all()) and bool((dw_out == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F16], ids=NAMES.get)
@pytest.mark.parametrize("T", [2, 30, 500])
def test_layouts(T, dtype):
    """Rows that are slices of wider ones at every alignment, weights with a pitch, transposed lists."""
    for pad in (1, 2, 4, 8):
        x, w_in, w_out, ids, weights, g, _ = layer(T, 4, 2, 96, 56, dtype, seed=pad, pad=pad)
        wide_in = torch.full((4, 112, 96 + pad), float("nan"), dtype=dtype, device="cuda")
        wide_out = torch.full((4, 96, 56 + pad), float("nan"), dtype=dtype, device="cuda")
        wide_in[:, :, :96], wide_out[:, :, :56] = w_in, w_out
        wide_g = torch.full((T, 96 + pad), float("nan"), dtype=dtype, device="cuda")
        wide_g[:, :96] = g
        args = (x, wide_in[:, :, :96], wide_out[:, :, :56], ids.t().contiguous().t(), weights.t().contiguous().t(), wide_g[:, :96])
        check(*args)
        shifted = [torch.empty(t.numel() + 1, dtype=dtype, device="cuda")[1:].view(t.shape).copy_(t) for t in (x, w_in, w_out, g)]
        check(shifted[0], shifted[1], shifted[2], ids, weights, shifted[3])


@pytest.mark.parametrize("dtype", [BF16, F16], ids=NAMES.get)
@pytest.mark.parametrize("T,E,D,F", [(1, 3, 1, 1), (5, 9, 3, 5), (2, 300, 15, 17), (40, 1024, 9, 34), (64, 12, 333, 90), (300, 5, 1001, 500),
                                     (9, 7, 530, 64), (9, 7, 64, 530)])
def test_weights_off_the_grid_give_the_bits_of_aligned_ones(T, E, D, F, dtype):
    """Every offset and odd pitches, NaN around the weights and in those of experts without rows:
    the copies that the products read hold the same elements as aligned weights."""
    lib = H.tg()
    x, w_in, w_out, ids, weights, g, _ = layer(T, E, 1, D, F, dtype, seed=D + F)
    ids %= max(1, E // 3)
    ids = E - 1 - 2 * ids  # from the last expert down, every second one
    idle = torch.ones(E, dtype=torch.bool, device="cuda")
    idle[ids.flatten()] = False
    w_in[idle], w_out[idle] = float("nan"), float("nan")

    def placed(w, lead, pad):
        rows, cols = w.shape[0] * w.shape[1], w.shape[2]
        buffer = torch.full((lead + rows * (cols + pad) + 64,), float("nan"), dtype=dtype, device="cuda")
        view = buffer.as_strided(w.shape, (w.shape[1] * (cols + pad), cols + pad, 1), lead)
        return view.copy_(w)

    def results(w_in, w_out):
        out, saved = lib.expert_mlp(x, w_in, w_out, ids, weights, save=True)
        got = [out, *lib.expert_mlp_backward(x, w_in, w_out, ids, weights, saved, g)]
        got += lib.expert_mlp_backward(x, w_in, w_out, ids, weights, saved, g, want_hidden=False)[1:]
        finished()
        return got

    want = results(placed(w_in, 0, -D % 8), placed(w_out, 0, -F % 8))
    Experts(x, w_in.nan_to_num(0), w_out.nan_to_num(0), ids, weights, g).check(**dict(zip(("out", "dx", "dw_in", "dw_out", "dw"), want)))
    for lead in range(8):
        for pad in (0, 1, 6):
            for a, b in zip(results(placed(w_in, lead, pad), placed(w_out, 7 - lead, pad)), want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("T,E,k", [(1, 6, 2), (3, 6, 2), (90, 6, 2), (40, 64, 40), (1, 64, 40)])
@pytest.mark.parametrize("D,F", [(97, 51), (104, 50), (101, 56), (7, 3)])
def test_odd_sizes_in_aligned_rows_and_many_picks(T, E, k, D, F):
    """Rows on the 16-byte grid whose last words are partly the next row's filling, which is NaN."""
    x, w_in, w_out, ids, weights, g, _ = layer(T, E, k, D, F, BF16, seed=D)
    nan = float("nan")
    ld, lf = (D + 7) // 8 * 8 + 8, (F + 7) // 8 * 8 + 8
    wide = [torch.full(s, nan, dtype=BF16, device="cuda") for s in ((T, ld), (E, 2 * F, ld), (E, D, lf), (T, ld))]
    for a, b in zip(wide, (x, w_in, w_out, g)):
        a[..., :b.shape[-1]] = b
    check(wide[0][:, :D], wide[1][:, :, :D], wide[2][:, :, :F], ids, weights, wide[3][:, :D])


def test_what_lies_beside_the_outputs_stays():
    """Through the C ABI, into rows with a pitch and guards; dx, dW and d_weights one at a time are the same bits."""
    lib = H.tg()
    T, E, k, D, F = 130, 5, 2, 200, 120
    x, w_in, w_out, ids, weights, g, _ = layer(T, E, k, D, F, BF16)
    _, want = both(x, w_in, w_out, ids, weights, g)
    s = torch.cuda.current_stream().cuda_stream
    saved = torch.empty(lib.experts_saved_size(T, E, k, D, F, lib.BF16)[1], dtype=torch.uint8, device="cuda")

    def lent(backward):
        n = lib.experts_workspace_size(backward, T, E, k, D, F, w_in.data_ptr(), D, w_out.data_ptr(), F, lib.BF16)[1]
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), n  # NaN, if it were read

    def wide(rows, cols, pad):
        return torch.full((rows + 2, cols + pad), 777.0, dtype=BF16, device="cuda")

    def same(buffer, cols, wanted):
        assert torch.equal(buffer[1:-1, :cols], wanted.reshape(-1, cols))
        assert bool((buffer[:, cols:] == 777.0).all()) and bool((buffer[0] == 777.0).all()) and bool((buffer[-1] == 777.0).all())

    for pad in (3, 8):
        out = wide(T, D, pad)
        ws, n = lent(False)
        assert lib.experts_forward(T, E, k, D, F, x.data_ptr(), D, w_in.data_ptr(), D, w_out.data_ptr(), F, ids.data_ptr(),
                                   weights.data_ptr(), lib.BF16, out[1].data_ptr(), D + pad, saved.data_ptr(), saved.numel(),
                                   None, ws.data_ptr(), n, s) == lib.OK
        same(out, D, want["out"])
        for keep in range(4):
            dx, dwi, dwo = wide(T, D, pad), wide(E * 2 * F, D, pad), wide(E * D, F, pad)
            dw = torch.full((T + 2, k), 777.0, device="cuda")
            ws, n = lent(True)
            p = [dx[1].data_ptr(), dwi[1].data_ptr(), dwo[1].data_ptr(), dw[1].data_ptr()]
            p = [v if i == keep else 0 for i, v in enumerate(p)]
            assert lib.experts_backward(T, E, k, D, F, x.data_ptr(), D, w_in.data_ptr(), D, w_out.data_ptr(), F,
                                        weights.data_ptr(), saved.data_ptr(), saved.numel(), g.data_ptr(), D, lib.BF16, p[0],
                                        D + pad, p[1], D + pad, p[2], F + pad, p[3], None, ws.data_ptr(), n, s) == lib.OK
            if keep == 0:
                same(dx, D, want["dx"])
            elif keep == 1:
                same(dwi, D, want["dw_in"])
            elif keep == 2:
                same(dwo, F, want["dw_out"])
            else:
                assert torch.equal(dw[1:-1], want["dw"]) and bool((dw[0] == 777.0).all()) and bool((dw[-1] == 777.0).all())
    finished()


@pytest.mark.parametrize("dtype", [BF16, F16], ids=NAMES.get)
def test_long_sums(dtype):
    """k axes of many chunks: D and F of 9000, an expert with 20000 rows of one sign."""
    check(*layer(70, 2, 1, 9000, 40, dtype)[:6])
    check(*layer(70, 2, 1, 64, 9000, dtype)[:6])
    x, w_in, w_out, ids, weights, g, _ = layer(20_000, 2, 1, 64, 32, dtype)
    ids.fill_(1)
    check(x.abs(), w_in.abs(), w_out.abs(), ids, weights, g.abs())


@pytest.mark.parametrize("size", [1e-6, 1e-4, 1.0, 1000.0])
def test_fp16_gradients_of_every_size(size):
    """dg and du are held in fp16 with the largest gradient at 16: neither small nor large ones are lost."""
    x, w_in, w_out, ids, weights, g, _ = layer(200, 4, 2, 128, 128, F16)
    check(x, w_in, w_out, ids, weights, (g.float() * 10 * size).half())


def test_bf16_values_of_every_size():
    """Rows whose results differ by many powers of two share 16-row blocks on their way to the join."""
    x, w_in, w_out, ids, weights, g, _ = layer(300, 3, 2, 128, 64, BF16)
    scale = torch.exp2(torch.randint(-12, 13, (300, 1), device="cuda").float())
    w_out = (w_out.float() * torch.exp2(torch.randint(-6, 7, (3, 128, 1), device="cuda").float())).bfloat16()
    check((x.float() * scale).bfloat16(), w_in, w_out, ids, weights, g)


def test_infinite_weights_stay_in_their_elements():
    """One infinite row of W_out makes one element of out infinite; the others are what they were."""
    x, w_in, w_out, ids, weights, g, _ = layer(100, 2, 1, 96, 64, BF16)
    lib = H.tg()
    want = lib.expert_mlp(x, w_in, w_out, ids, weights, save=True)[0]
    w_out[:, 17, 3] = float("inf")
    for save in (False, True):
        got = lib.expert_mlp(x, w_in, w_out, ids, weights, save=save)[0]
        assert not bool(got[:, 17].isfinite().any())
        keep = torch.arange(96, device="cuda") != 17
        assert torch.equal(got[:, keep], want[:, keep])


def test_gradients_against_differences():
    """Central differences of the 64-bit definition along random directions, the library's gradients against them."""
    x, w_in, w_out, ids, weights, g, gen = layer(60, 4, 2, 48, 40, BF16)
    _, got = both(x, w_in, w_out, ids, weights, g)
    ref = Experts(x, w_in, w_out, ids, weights, g)

    def value(a, b, c, w):
        out = torch.zeros(60, 48, dtype=torch.float64, device="cuda")
        for e in range(4):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            gu = a[t] @ b[e].t()
            out.index_add_(0, t, w[t, j][:, None] * ((torch.nn.functional.silu(gu[:, :40]) * gu[:, 40:]) @ c[e].t()))
        return (out * g.double()).sum()

    args = [x.double(), w_in.double(), w_out.double(), weights.double()]
    for i, name in enumerate(("dx", "dw_in", "dw_out", "dw")):
        step = torch.randn(args[i].shape, dtype=torch.float64, device="cuda", generator=gen)
        up, down = list(args), list(args)
        h = 1e-5
        up[i], down[i] = args[i] + h * step, args[i] - h * step
        slope = float((value(*up) - value(*down)) / (2 * h))
        # what the elementwise bounds allow, and the differences' own error (h^2 and 2^-53 / h of the terms)
        room = float((getattr(ref, "e_" + name) * step.abs()).sum()) + 1e-6 * float((getattr(ref, name) * step).abs().sum())
        assert abs(float((got[name].double() * step).sum()) - slope) <= room, name


@pytest.mark.parametrize("T", [1, 40, 500])
def test_gradients_through_torch(T):
    lib = H.tg()
    x, w_in, w_out, ids, weights, g, _ = layer(T, 5, 2, 64, 48, BF16)
    _, want = both(x, w_in, w_out, ids, weights, g)
    leaves = [t.clone().requires_grad_() for t in (x, w_in, w_out, weights)]
    out, saved = lib.expert_mlp(leaves[0], leaves[1], leaves[2], ids, leaves[3])
    assert out.requires_grad and not saved.requires_grad and torch.equal(out, want["out"])
    out.backward(g)
    for leaf, name in zip(leaves, ("dx", "dw_in", "dw_out", "dw")):
        assert torch.equal(leaf.grad, want[name]), name
    # one of them alone, with an expanded gradient (that of a sum)
    leaf = w_out.clone().requires_grad_()
    lib.expert_mlp(x, w_in, leaf, ids, weights)[0].sum().backward()
    again = lib.expert_mlp_backward(x, w_in, w_out, ids, weights, lib.expert_mlp(x, w_in, w_out, ids, weights, save=True)[1],
                                    torch.ones_like(g), want_hidden=False, want_in=False, want_weights=False)
    assert torch.equal(leaf.grad, again[2]) and again[0] is again[1] is again[3] is None
    with torch.no_grad():
        assert lib.expert_mlp(leaves[0], leaves[1], leaves[2], ids, leaves[3])[1] is None


@pytest.mark.parametrize("T,dtype", [(1, BF16), (40, F16), (700, BF16), (3000, F16)])
def test_a_captured_layer_replays(T, dtype):
    """Routing, products, gradients and their clipping in one graph: replayed on new inputs they give plain calls' bits."""
    lib = H.tg()
    E, k, D, F = 8, 2, 64, 48
    x, w_in, w_out, _, _, g, gen = layer(T, E, k, D, F, dtype)
    logits = torch.randn(T, E, device="cuda", generator=gen)
    logits[T // 2] = -math.inf

    def step():
        ids, weights = lib.route_experts(logits, k)
        short = lib.expert_mlp(x, w_in, w_out, ids, weights)[0]
        out, saved = lib.expert_mlp(x, w_in, w_out, ids, weights, save=True)
        dx, dw_in, dw_out, dw = lib.expert_mlp_backward(x, w_in, w_out, ids, weights, saved, g)
        d_logits = lib.route_experts_backward(logits, ids, dw)
        grads = [dw_in, dw_out]
        norm = lib.clip_gradients(grads, 0.5)
        return ids, weights, short, out, dx, d_logits, *grads, norm

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (2, 3):
        logits.copy_(torch.randn(T, E, device="cuda", generator=gen))
        x.copy_(layer(T, E, k, D, F, dtype, seed=seed)[0])
        graph.replay()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    finished()


def test_another_stream_and_lent_workspaces():
    lib = H.tg()
    x, w_in, w_out, ids, weights, g, _ = layer(300, 4, 2, 64, 48, BF16)
    plain, want = both(x, w_in, w_out, ids, weights, g)
    side = torch.cuda.Stream()
    sizes = (300, 4, 2, 64, 48)
    n = [lib.experts_workspace_size(b, *sizes, 0, 64, 0, 48, lib.BF16)[1] for b in (False, True)]
    ws = [torch.full((v + 100,), 255, dtype=torch.uint8, device="cuda") for v in n]
    torch.cuda.synchronize()
    out, saved = lib.expert_mlp(x, w_in, w_out, ids, weights, save=True, workspace=ws[0], stream=side.cuda_stream)
    got = lib.expert_mlp_backward(x, w_in, w_out, ids, weights, saved, g, workspace=ws[1], stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, want["out"])
    for a, name in zip(got, ("dx", "dw_in", "dw_out", "dw")):
        assert torch.equal(a, want[name])
    with pytest.raises(ValueError, match="workspace"):
        lib.expert_mlp(x, w_in, w_out, ids, weights, save=True, workspace=ws[0][:n[0] - 1])


def test_two_calls_at_once():
    """Two streams, each with its own workspace: neither changes the other's bits."""
    lib = H.tg()
    layers = [layer(900, 6, 2, 256, 128, BF16, seed=s) for s in (1, 2)]
    want = [both(*a[:6])[1] for a in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for a, s in zip(layers, streams):
            out, saved = lib.expert_mlp(*a[:5], save=True, stream=s.cuda_stream)
            got.append((out, saved) + lib.expert_mlp_backward(*a[:5], saved, a[5], stream=s.cuda_stream))
        torch.cuda.synchronize()
        for w, (out, _, dx, dw_in, dw_out, dw) in zip(want, got):
            for x, name in ((out, "out"), (dx, "dx"), (dw_in, "dw_in"), (dw_out, "dw_out"), (dw, "dw")):
                assert torch.equal(x, w[name]), name
    finished()


def test_waits_that_run_out_are_reported():
    """A bound of a microsecond on every wait: the calls give up or finish, the next ones are whole."""
    lib = H.tg()
    T, E, k, D, F = 600, 3, 2, 512, 256
    x, w_in, w_out, ids, weights, g, _ = layer(T, E, k, D, F, BF16)
    s = torch.cuda.current_stream().cuda_stream
    saved = torch.empty(lib.experts_saved_size(T, E, k, D, F, lib.BF16)[1], dtype=torch.uint8, device="cuda")
    n = lib.experts_workspace_size(False, T, E, k, D, F, w_in.data_ptr(), D, w_out.data_ptr(), F, lib.BF16)[1]
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(x)
    assert lib.experts_forward(T, E, k, D, F, x.data_ptr(), D, w_in.data_ptr(), D, w_out.data_ptr(), F, ids.data_ptr(),
                               weights.data_ptr(), lib.BF16, out.data_ptr(), D, saved.data_ptr(), saved.numel(),
                               {"wait_timeout_us": 1}, ws.data_ptr(), n, s) == lib.OK
    assert lib.device_status(s) in (lib.OK, lib.ERR_DEVICE_TIMEOUT)
    check(x, w_in, w_out, ids, weights, g)


def test_refusals():
    lib = H.tg()
    x, w_in, w_out, ids, weights, g, _ = layer(20, 4, 2, 64, 48, BF16)
    out, saved = lib.expert_mlp(x, w_in, w_out, ids, weights, save=True)
    for args in ((x.float(), w_in, w_out, ids, weights), (x, w_in[:, :-1], w_out, ids, weights), (x, w_in.half(), w_out, ids, weights),
                 (x, w_in, w_out[:, :-1], ids, weights), (x, w_in, w_out, ids.int(), weights), (x, w_in, w_out, ids, weights.half()),
                 (x, w_in, w_out, ids[:-1], weights), (x, w_in, w_out, ids, weights[:, :1]), (x.cpu(), w_in, w_out, ids, weights),
                 (x, w_in.cpu(), w_out, ids, weights), (x.t(), w_in, w_out, ids, weights), (x, w_in[::2], w_out[::2], ids, weights),
                 (x, w_in.transpose(1, 2), w_out, ids, weights), (x[0], w_in, w_out, ids, weights)):
        with pytest.raises(ValueError):
            lib.expert_mlp(*args)
    for more in ({"saved": None}, {"saved": saved[:-1]}, {"grad_out": g.half()}, {"grad_out": g[:-1]}, {"grad_out": g.cpu()}):
        args = {"saved": saved, "grad_out": g, **more}
        with pytest.raises(ValueError):
            lib.expert_mlp_backward(x, w_in, w_out, ids, weights, **args)
    # a transposed gradient is made dense, as torch's backward passes hand them over
    t = g.t().contiguous().t()
    for a, b in zip(lib.expert_mlp_backward(x, w_in, w_out, ids, weights, saved, t),
                    lib.expert_mlp_backward(x, w_in, w_out, ids, weights, saved, g)):
        assert torch.equal(a, b)
