"""The vocabulary-head losses on the GPU against their definition in 64 bits
(tests/loss_reference.py), at the sizes, lists and masks where they can go
wrong, through the tensor functions and through the C ABI."""
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


def head(T, V, D, dtype, seed=0, pad_h=0, pad_w=0, spread=2.0):
    """Hidden states and a weight whose logits spread with a deviation of about `spread`."""
    gen = torch.Generator(device="cuda").manual_seed(1000 + seed)
    h = torch.randn(T, D + pad_h, device="cuda", generator=gen).to(dtype)
    w = (torch.randn(V, D + pad_w, device="cuda", generator=gen) * (spread / math.sqrt(D))).to(dtype)
    return h[:, :D], w[:, :D], gen


def targets_for(T, V, gen, ignored=0.0):
    y = torch.randint(0, V, (T,), device="cuda", generator=gen)
    if ignored:
        y[torch.rand(T, device="cuda", generator=gen) < ignored] = -100
    return y


def lists_for(T, V, K, gen, dtype=F32):
    ids = torch.randint(0, V, (T, K), device="cuda", generator=gen)  # entries may repeat: masses add
    logits = 4 * torch.randn(T, K, device="cuda", generator=gen)
    return ids, logits.to(dtype)


def finished():
    lib = H.tg()
    assert lib.device_status(torch.cuda.current_stream().cuda_stream) == lib.OK
    return lib


def xent_both(h, w, y, g, **more):
    lib = H.tg()
    loss, lse = lib.linear_cross_entropy(h, w, y, **more)
    dh, dw = lib.linear_cross_entropy_backward(h, w, y, lse, g, **more)
    finished()
    return {"loss": loss, "lse": lse, "dh": dh, "dw": dw}


def distill_both(h, w, ids, logits, g, **more):
    lib = H.tg()
    loss, lse = lib.linear_distillation(h, w, ids, logits, **more)
    dh, dw = lib.linear_distillation_backward(h, w, ids, logits, lse, g, **more)
    finished()
    return {"loss": loss, "lse": lse, "dh": dh, "dw": dw}


SHAPES = [
    (1, 1, 1), (1, 2, 8), (1, 1000, 64), (2, 255, 7), (3, 257, 33), (31, 256, 64), (33, 513, 65), (64, 4096, 128),
    (127, 1031, 200), (128, 300, 511), (129, 2049, 96), (255, 777, 320), (256, 512, 256), (257, 1280, 257),
    (300, 5003, 333), (511, 263, 1000), (700, 1031, 512), (1000, 1500, 1001),
]


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,D", SHAPES)
def test_xent_matches_its_definition(T, V, D, dtype):
    h, w, gen = head(T, V, D, dtype, seed=T + V)
    y = targets_for(T, V, gen)
    g = torch.full((T,), 1.0 / T, device="cuda")
    ref.xent(h, w, y, g=g).check(**xent_both(h, w, y, g))


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,D,K", [(1, 300, 64, 1), (1, 5, 8, 5), (7, 1000, 33, 3), (64, 4096, 128, 64),
                                     (130, 513, 72, 17), (257, 1031, 200, 32), (300, 257, 96, 256), (513, 2000, 512, 100)])
def test_distillation_matches_its_definition(T, V, D, K, dtype):
    h, w, gen = head(T, V, D, dtype, seed=T + K)
    ids, logits = lists_for(T, V, K, gen)
    g = torch.rand(T, device="cuda", generator=gen) / T
    ref.distill(h, w, ids, logits, 2.0, g).check(**distill_both(h, w, ids, logits, g, temperature=2.0))


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,D,ignored", [(40, 700, 64, 0.5), (300, 1000, 130, 0.9), (600, 513, 256, 0.3),
                                           (513, 300, 72, 0.02)])
def test_ignored_rows_cost_nothing_whatever_they_hold(T, V, D, ignored, dtype):
    """NaN and infinities in ignored rows reach no output; weighted gradients, smoothing and z-loss."""
    h, w, gen = head(T, V, D, dtype, seed=T, pad_h=5)
    y = targets_for(T, V, gen, ignored)
    y[0] = -100
    dead = y == -100
    h[dead] = float("nan")
    h[0] = float("inf")
    g = torch.randn(T, device="cuda", generator=gen) / T
    g[dead] = float("nan")
    more = {"scale": 0.7, "z_loss": 1e-2}
    got = xent_both(h, w, y, g, label_smoothing=0.1, **more)
    ref.xent(h, w, y, smoothing=0.1, g=g, **more).check(**got)
    for name in ("loss", "lse", "dh"):
        assert bool((got[name][dead] == 0).all()), name


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
def test_lists_of_every_kind(dtype):
    """Unused places, empty rows, masses of 0, rows that are all -inf, the type's lowest value, repeated entries."""
    T, V, D, K = 300, 900, 100, 12
    h, w, gen = head(T, V, D, dtype, seed=3)
    ids, logits = lists_for(T, V, K, gen)
    ids[torch.rand(T, K, device="cuda", generator=gen) < 0.4] = -1
    ids[5] = -1
    ids[6] = -7
    ids[7] = 3
    ids[8] = torch.arange(K, device="cuda")
    logits[8] = float("-inf")
    logits[8, 4] = 1.0
    ids[9] = torch.arange(K, device="cuda")
    logits[9] = float("-inf")
    ids[10] = torch.arange(K, device="cuda")
    logits[10, 1:] = torch.finfo(F32).min
    ids[11, 0] = 2
    logits[11, 1:] = float("-inf")
    logits[ids < 0] = float("nan")  # an unused place's logit is not read into anything
    h[5:7] = float("nan")
    h[9] = float("nan")
    g = torch.rand(T, device="cuda", generator=gen)
    got = distill_both(h, w, ids, logits, g)
    ref.distill(h, w, ids, logits.nan_to_num(nan=0.0, neginf=float("-inf")), 1.0, g).check(**got)
    for row in (5, 6, 9):
        assert float(got["loss"][row]) == 0.0 and bool((got["dh"][row] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [1, 3, 300])
def test_no_row_counts(T, dtype):
    V, D = 700, 96
    h, w, _ = head(T, V, D, dtype)
    h[:] = float("nan")
    y = torch.full((T,), 7, device="cuda")
    got = xent_both(h, w, y, torch.ones(T, device="cuda"), ignore_index=7)
    for name, x in got.items():
        assert bool((x == 0).all()), name
    got = distill_both(h, w, torch.full((T, 3), -1, device="cuda"), torch.zeros(T, 3, device="cuda"),
                       torch.ones(T, device="cuda"))
    for name, x in got.items():
        assert bool((x == 0).all()), name


def test_no_rows_at_all():
    lib = H.tg()
    h, w, _ = head(0, 300, 64, BF16)
    y = torch.zeros(0, dtype=torch.int64, device="cuda")
    loss, lse = lib.linear_cross_entropy(h, w, y)
    assert loss.numel() == lse.numel() == 0
    dh, dw = lib.linear_cross_entropy_backward(h, w, y, lse, torch.zeros(0, device="cuda"))
    finished()
    assert dh.shape == (0, 64) and bool((dw == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
def test_data_errors_give_nan_and_no_gradient(dtype):
    T, V, D = 40, 500, 64
    h, w, gen = head(T, V, D, dtype)
    y = targets_for(T, V, gen)
    wrong = [3, 17, 39]
    z = y.clone()
    z[3], z[17], z[39] = V, -1, 1 << 40
    y[wrong] = -100
    g = torch.ones(T, device="cuda")
    got = xent_both(h, w, z, g)
    assert bool(torch.isnan(got["loss"][wrong]).all())
    for name in ("loss", "lse"):
        got[name][wrong] = 0
    ref.xent(h, w, y, g=g).check(**got)
    ids, logits = lists_for(T, V, 5, gen)
    wild = ids.clone()
    wild[4, 2] = V
    ids[4] = -1
    got = distill_both(h, w, wild, logits, g)
    assert math.isnan(float(got["loss"][4]))
    got["loss"][4] = got["lse"][4] = 0
    ref.distill(h, w, ids, logits, 1.0, g).check(**got)


@pytest.mark.parametrize("pad_h,pad_w,D", [(8, 8, 64), (1, 0, 64), (0, 1, 64), (4, 2, 100), (3, 4, 77)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
def test_row_strides_and_alignments(pad_h, pad_w, D, dtype):
    T, V = 200, 1100
    h, w, gen = head(T, V, D, dtype, pad_h=pad_h, pad_w=pad_w)
    y = targets_for(T, V, gen, 0.2)
    g = torch.rand(T, device="cuda", generator=gen)
    ref.xent(h, w, y, g=g).check(**xent_both(h, w, y, g))
    ids, logits = lists_for(T, V, 9, gen)
    wide = torch.full((T, 13), 5, device="cuda")
    wide[:, :9] = ids
    tall = torch.zeros(T, 11, device="cuda")
    tall[:, :9] = logits
    ref.distill(h, w, ids, logits, 1.0, g).check(**distill_both(h, w, wide[:, :9], tall[:, :9], g))


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("piece", [256, 768, 4096])
@pytest.mark.parametrize("pad_w", [0, 1])
def test_pieces_of_the_vocabulary(piece, pad_w, dtype):
    """Targets on both sides of the pieces' borders; the last piece ends inside a tile."""
    T, V, D = 270, 2500, 136
    h, w, gen = head(T, V, D, dtype, pad_w=pad_w)
    y = targets_for(T, V, gen, 0.1)
    for i, v in enumerate([0, 255, 256, 257, 511, 512, 767, 768, 1023, 1024, V - 1, 2303, 2304]):
        y[i] = v
    g = torch.rand(T, device="cuda", generator=gen)
    ref.xent(h, w, y, smoothing=0.2, g=g).check(**xent_both(h, w, y, g, label_smoothing=0.2, piece=piece))
    ids, logits = lists_for(T, V, 40, gen)
    ref.distill(h, w, ids, logits, 1.5, g).check(**distill_both(h, w, ids, logits, g, temperature=1.5, piece=piece))


@pytest.mark.parametrize("dtype,code", [(BF16, 2), (F16, 1), (F32, 0)], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 0), (8, 1), (1, 3)])
def test_c_abi_writes_only_its_outputs(dtype, code, pad, offset):
    """dH and dW with row pitches and offsets of their own: what lies between the rows stays as it was."""
    lib = H.tg()
    T, V, D = 150, 600, 88
    h, w, gen = head(T, V, D, dtype)
    y = targets_for(T, V, gen, 0.2)
    g = torch.rand(T, device="cuda", generator=gen)
    loss, lse = lib.linear_cross_entropy(h, w, y)
    ld = D + pad
    outs = []
    for rows in (T, V):
        flat = torch.full((offset + rows * ld + 64,), -77.0, dtype=dtype, device="cuda")
        outs.append((flat, flat[offset:offset + rows * ld].view(rows, ld)))
    st, need = lib.loss_workspace_size(True, T, V, D, 0, w.data_ptr(), D, code)
    assert st == lib.OK
    ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    es = h.element_size()
    st = lib.xent_backward(T, V, D, h.data_ptr(), D, w.data_ptr(), D, y.data_ptr(), lse.data_ptr(), g.data_ptr(), code,
                           outs[0][0].data_ptr() + offset * es, ld, outs[1][0].data_ptr() + offset * es, ld, None,
                           ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert st == lib.OK, lib.status_string(st)
    finished()
    assert bool((ws[need:] == 0xA5).all()), "written past the workspace"
    ref.xent(h, w, y, g=g).check(loss=loss, lse=lse, dh=outs[0][1][:, :D], dw=outs[1][1][:, :D])
    for (flat, view), rows in zip(outs, (T, V)):
        assert bool((view[:, D:] == -77).all()) and bool((flat[:offset] == -77).all())
        assert bool((flat[offset + rows * ld:] == -77).all())


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
def test_one_gradient_alone_is_the_same(dtype):
    lib = H.tg()
    h, w, gen = head(200, 900, 128, dtype)
    y = targets_for(200, 900, gen, 0.2)
    g = torch.rand(200, device="cuda", generator=gen)
    _, lse = lib.linear_cross_entropy(h, w, y)
    dh, dw = lib.linear_cross_entropy_backward(h, w, y, lse, g)
    a, none = lib.linear_cross_entropy_backward(h, w, y, lse, g, want_weight=False)
    assert none is None and torch.equal(a, dh)
    none, b = lib.linear_cross_entropy_backward(h, w, y, lse, g, want_hidden=False)
    assert none is None and torch.equal(b, dw)
    finished()


@pytest.mark.parametrize("T,V,D", [(4, 20000, 256), (700, 3000, 512)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_same_bits_every_time(T, V, D, dtype):
    h, w, gen = head(T, V, D, dtype)
    ids, logits = lists_for(T, V, 20, gen)
    g = torch.rand(T, device="cuda", generator=gen)
    first = distill_both(h, w, ids, logits, g)
    for _ in range(3):
        again = distill_both(h, w, ids, logits, g)
        for name in first:
            assert torch.equal(first[name], again[name]), name


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
def test_sizes_of_upstream_gradients(dtype):
    """Gradients far from 1, negative, zero, and of very different sizes keep their relative accuracy."""
    T, V, D = 90, 700, 96
    h, w, gen = head(T, V, D, dtype)
    y = targets_for(T, V, gen)
    top = {BF16: 1e20, F16: 1e2, F32: 1e20}[dtype]
    for size in (top, 1.0, 1e-3):
        g = size * torch.randn(T, device="cuda", generator=gen)
        g[:5] = 0
        g[5:20] *= 1e-3
        r = ref.xent(h, w, y, g=g)
        got = xent_both(h, w, y, g)
        r.check(**got)
        assert bool((got["dh"][:5] == 0).all())
    got = xent_both(h, w, y, torch.zeros(T, device="cuda"))
    assert bool((got["dh"] == 0).all()) and bool((got["dw"] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
def test_large_logits(dtype):
    """Logits of several hundred: the running maximum keeps the exponentials in range."""
    T, V, D = 70, 1500, 64
    h, w, gen = head(T, V, D, dtype, spread=150.0)
    y = targets_for(T, V, gen)
    g = torch.ones(T, device="cuda")
    ref.xent(h, w, y, g=g).check(**xent_both(h, w, y, g))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_nan_and_infinity_stay_in_their_rows(dtype):
    lib = H.tg()
    T, V, D = 300, 600, 64
    h, w, gen = head(T, V, D, dtype)
    y = targets_for(T, V, gen)
    clean, clean_lse = lib.linear_cross_entropy(h, w, y)
    h2 = h.clone()
    h2[10, 3] = float("nan")
    h2[20, 5] = float("inf")
    loss, lse = lib.linear_cross_entropy(h2, w, y)
    finished()
    assert math.isnan(float(loss[10])) and not math.isfinite(float(loss[20]))
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[10] = rest[20] = False
    assert torch.equal(loss[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])


@pytest.mark.parametrize("kind", ["xent", "distill"])
def test_gradient_against_differences(kind):
    """fp32: (L(x + e d) - L(x - e d)) / 2e against <gradient, d> for a weighted
    sum of losses.  With e = 2^-6 and |d| of the size of x, the third-order term
    is below 1e-3 of the slope's scale and the losses' roundings, 2^-20 * 12 /
    2e, below 1e-3: the slopes agree to 1e-2 of the gradient's norm."""
    lib = H.tg()
    T, V, D = 60, 800, 64
    h, w, gen = head(T, V, D, F32, spread=1.0)
    y = targets_for(T, V, gen, 0.2)
    ids, logits = lists_for(T, V, 8, gen)
    g = torch.rand(T, device="cuda", generator=gen)

    def value(h, w):
        loss = (lib.linear_cross_entropy(h, w, y, label_smoothing=0.1, z_loss=1e-3) if kind == "xent" else
                lib.linear_distillation(h, w, ids, logits, temperature=1.3))[0]
        return float((g.double() * loss.double()).sum())

    if kind == "xent":
        _, lse = lib.linear_cross_entropy(h, w, y, label_smoothing=0.1, z_loss=1e-3)
        dh, dw = lib.linear_cross_entropy_backward(h, w, y, lse, g, label_smoothing=0.1, z_loss=1e-3)
    else:
        _, lse = lib.linear_distillation(h, w, ids, logits, temperature=1.3)
        dh, dw = lib.linear_distillation_backward(h, w, ids, logits, lse, g, temperature=1.3)
    e = 2.0 ** -6
    for x, grad, at in ((h, dh, 0), (w, dw, 1)):
        d = grad / grad.norm() * x.norm() * 0.05  # along the gradient: the slope is its norm times |d|
        up = value(*((x + e * d, w) if at == 0 else (h, x + e * d)))
        down = value(*((x - e * d, w) if at == 0 else (h, x - e * d)))
        slope = float((grad.double() * d.double()).sum())
        assert abs((up - down) / (2 * e) - slope) <= 1e-2 * abs(slope)


def test_on_another_stream():
    lib = H.tg()
    h, w, gen = head(300, 2000, 128, BF16)
    ids, logits = lists_for(300, 2000, 16, gen, dtype=BF16)
    g = torch.rand(300, device="cuda", generator=gen)
    want = distill_both(h, w, ids, logits, g)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    loss, lse = lib.linear_distillation(h, w, ids, logits, stream=side.cuda_stream)
    dh, dw = lib.linear_distillation_backward(h, w, ids, logits, lse, g, stream=side.cuda_stream)
    assert lib.device_status(side.cuda_stream) == lib.OK
    for name, x in (("loss", loss), ("lse", lse), ("dh", dh), ("dw", dw)):
        assert torch.equal(x, want[name]), name


def test_offsets_past_32_bits():
    """A weight of more than 2^32 bytes and 2^31 elements: its last rows are read and written."""
    lib = H.tg()
    T, V, D = 3, 1 << 20, 2064
    assert V * D > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(5)
    w = torch.empty(V, D, dtype=BF16, device="cuda")
    for lo in range(0, V, 1 << 16):
        w[lo:lo + (1 << 16)] = (torch.randn(1 << 16, D, device="cuda", generator=gen) / math.sqrt(D)).to(BF16)
    h = torch.randn(T, D, device="cuda", generator=gen).to(BF16)
    y = torch.tensor([V - 1, V - 300, 5], device="cuda")
    g = torch.tensor([1.0, 2.0, 0.5], device="cuda")
    loss, lse = lib.linear_cross_entropy(h, w, y)
    dh, dw = lib.linear_cross_entropy_backward(h, w, y, lse, g)
    finished()
    z = torch.cat([h.double() @ w[lo:lo + (1 << 16)].double().t() for lo in range(0, V, 1 << 16)], dim=1)
    want = torch.logsumexp(z, dim=1)
    assert float((lse.double() - want).abs().max()) < 1e-4
    assert float((loss.double() - (want - z.gather(1, y[:, None])[:, 0])).abs().max()) < 1e-4
    dz = torch.exp(z - want[:, None])
    dz.scatter_add_(1, y[:, None], torch.full((T, 1), -1.0, dtype=torch.float64, device="cuda"))
    dz *= g.double()[:, None]
    for rows in (slice(V - 512, V), slice(0, 64)):
        ref_dw = dz[:, rows].t() @ h.double()
        bound = 2.0 ** -7 * (dz[:, rows].abs().t() @ h.double().abs())
        assert bool(((dw[rows].double() - ref_dw).abs() <= bound).all())
    ref_dh = sum(dz[:, lo:lo + (1 << 16)] @ w[lo:lo + (1 << 16)].double() for lo in range(0, V, 1 << 16))
    size = sum(dz[:, lo:lo + (1 << 16)].abs() @ w[lo:lo + (1 << 16)].double().abs() for lo in range(0, V, 1 << 16))
    assert bool(((dh.double() - ref_dh).abs() <= 2.0 ** -7 * size).all())


def test_device_side_timeout_is_not_left_behind():
    """A generous bound on the waits changes nothing and leaves no status."""
    lib = H.tg()
    h, w, gen = head(64, 1000, 64, BF16)
    y = targets_for(64, 1000, gen)
    lse = torch.empty(64, device="cuda")
    loss = torch.empty(64, device="cuda")
    st, need = lib.loss_workspace_size(False, 64, 1000, 64, 0, w.data_ptr(), 64, lib.BF16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    opts = lib.LossOptions(ignore_index=-100, wait_timeout_us=5000000)
    st = lib.xent_forward(64, 1000, 64, h.data_ptr(), 64, w.data_ptr(), 64, y.data_ptr(), lib.BF16, loss.data_ptr(),
                          lse.data_ptr(), opts, ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert st == lib.OK
    finished()
    ref.xent(h, w, y).check(loss=loss, lse=lse)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 9, 16, 31, 32, 33])
@pytest.mark.parametrize("D,left,right", [(64, 0, 0), (40, 1, 0), (41, 0, 0), (37, 3, 2), (50, 2, 4), (515, 5, 1)])
def test_few_rows_beside_nan(T, D, left, right, dtype):
    """Rows of W at every offset from the 16-byte grid, inside a matrix whose other columns are NaN."""
    lib = H.tg()
    V = 777
    gen = torch.Generator(device="cuda").manual_seed(T * 1000 + D)
    whole = torch.full((V + 2, left + D + right), float("nan"), dtype=dtype, device="cuda")
    w = whole[1:V + 1, left:left + D]
    w.copy_((torch.randn(V, D, device="cuda", generator=gen) * (2.0 / math.sqrt(D))).to(dtype))
    wide = torch.full((T, D + left), float("nan"), dtype=dtype, device="cuda")
    h = wide[:, left:]
    h.copy_(torch.randn(T, D, device="cuda", generator=gen).to(dtype))
    y = targets_for(T, V, gen, 0.2)
    loss, lse = lib.linear_cross_entropy(h, w, y, label_smoothing=0.1, z_loss=1e-3)
    ref.xent(h, w, y, smoothing=0.1, z_loss=1e-3).check(loss=loss, lse=lse)
    ids, logits = lists_for(T, V, 7, gen)
    loss, lse = lib.linear_distillation(h, w, ids, logits)
    finished()
    ref.distill(h, w, ids, logits).check(loss=loss, lse=lse)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("V,D,left,right", [(777, 64, 0, 0), (5, 41, 0, 0), (33, 50, 2, 4), (777, 1030, 0, 2),
                                            (300, 2100, 4, 0), (257, 37, 3, 2)])
def test_few_rows_gradients_beside_nan(T, V, D, left, right, dtype):
    """Less than a share of entries, columns past one block's, rows that do not count; the rest of the matrix NaN."""
    gen = torch.Generator(device="cuda").manual_seed(T * 1000 + D)
    whole = torch.full((V + 2, left + D + right), float("nan"), dtype=dtype, device="cuda")
    w = whole[1:V + 1, left:left + D]
    w.copy_((torch.randn(V, D, device="cuda", generator=gen) * (2.0 / math.sqrt(D))).to(dtype))
    wide = torch.full((T, D + left), float("nan"), dtype=dtype, device="cuda")
    h = wide[:, left:]
    h.copy_(torch.randn(T, D, device="cuda", generator=gen).to(dtype))
    y = targets_for(T, V, gen)
    g = torch.randn(T, device="cuda", generator=gen)
    if T > 2:
        y[1] = -100
        h[1] = g[1] = float("nan")
    more = {"scale": 0.8, "z_loss": 1e-2}
    ref.xent(h, w, y, smoothing=0.1, g=g, **more).check(**xent_both(h, w, y, g, label_smoothing=0.1, **more))
    ids, logits = lists_for(T, V, 7, gen)
    if T > 2:
        ids[1] = -1
    ref.distill(h, w, ids, logits, 2.0, g).check(**distill_both(h, w, ids, logits, g, temperature=2.0))


@pytest.mark.parametrize("T", [7, 9, 16, 17, 31, 32])
@pytest.mark.parametrize("V,D,left,right", [(16384, 64, 0, 0), (16641, 37, 3, 2), (20000, 1, 0, 3), (17000, 130, 0, 2),
                                            (300, 5300, 4, 0)])
def test_tens_of_fp32_rows_beside_nan(T, V, D, left, right):
    """Large vocabularies (and rows too long for shared memory), whole and in pieces; the rest of the matrix NaN."""
    lib = H.tg()
    gen = torch.Generator(device="cuda").manual_seed(T * 1000 + D)
    whole = torch.full((V + 2, left + D + right), float("nan"), device="cuda")
    w = whole[1:V + 1, left:left + D]
    w.copy_(torch.randn(V, D, device="cuda", generator=gen) * (2.0 / math.sqrt(D)))
    wide = torch.full((T, D + left), float("nan"), device="cuda")
    h = wide[:, left:]
    h.copy_(torch.randn(T, D, device="cuda", generator=gen))
    y = targets_for(T, V, gen)
    y[:3] = torch.tensor([V - 1, 0, 255], device="cuda").clamp(max=V - 1)
    y[3] = -100
    h[3] = float("inf")
    for piece in (0, 768):
        loss, lse = lib.linear_cross_entropy(h, w, y, label_smoothing=0.1, z_loss=1e-3, piece=piece)
        finished()
        ref.xent(h, w, y, smoothing=0.1, z_loss=1e-3).check(loss=loss, lse=lse)
        assert float(loss[3]) == float(lse[3]) == 0
    ids, logits = lists_for(T, V, 40, gen)
    ids[3] = -1
    ids[4, 1:4] = ids[4, 0]
    loss, lse = lib.linear_distillation(h, w, ids, logits)
    finished()
    ref.distill(h, w, ids, logits).check(loss=loss, lse=lse)


@pytest.mark.parametrize("dtype,code,T", [(BF16, 2, 2), (F16, 1, 1), (F32, 0, 5)], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad_w", [0, 1])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 0), (8, 1), (2, 2)])
def test_few_rows_write_only_their_outputs(dtype, code, T, pad_w, pad, offset):
    lib = H.tg()
    V, D = 601, 90
    h, w, gen = head(T, V, D + pad_w, dtype)
    D += pad_w
    y = targets_for(T, V, gen)
    g = torch.rand(T, device="cuda", generator=gen)
    loss, lse = lib.linear_cross_entropy(h, w, y)
    ld = D + pad
    es = h.element_size()
    st, need = lib.loss_workspace_size(True, T, V, D, 0, w.data_ptr(), D, code)
    assert st == lib.OK
    for want in ((True, True), (True, False), (False, True)):
        outs = []
        for rows in (T, V):
            flat = torch.full((offset + rows * ld + 64,), -77.0, dtype=dtype, device="cuda")
            outs.append((flat, flat[offset:offset + rows * ld].view(rows, ld)))
        ptrs = [o[0].data_ptr() + offset * es if on else 0 for o, on in zip(outs, want)]
        ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        st = lib.xent_backward(T, V, D, h.data_ptr(), D, w.data_ptr(), D, y.data_ptr(), lse.data_ptr(), g.data_ptr(),
                               code, ptrs[0], ld, ptrs[1], ld, None, ws.data_ptr(), need,
                               torch.cuda.current_stream().cuda_stream)
        assert st == lib.OK, lib.status_string(st)
        finished()
        assert bool((ws[need:] == 0xA5).all()), "written past the workspace"
        if all(want):
            first = [o[1][:, :D].clone() for o in outs]
            ref.xent(h, w, y, g=g).check(loss=loss, lse=lse, dh=first[0], dw=first[1])
        for (flat, view), rows, on, both in zip(outs, (T, V), want, first):
            if not on:
                assert bool((flat == -77).all())
                continue
            assert torch.equal(view[:, :D], both)
            assert bool((view[:, D:] == -77).all()) and bool((flat[:offset] == -77).all())
            assert bool((flat[offset + rows * ld:] == -77).all())


def test_few_rows_gradients_past_32_bits():
    """A weight of more than 2^31 elements; its end alone gives the same bits, dH is the formula's."""
    lib = H.tg()
    T, V, D, last = 2, 140_000, 16_384, 600
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough free memory")
    h, w, gen = head(T, V, D, BF16)
    y = torch.tensor([V - 1, V - last], device="cuda")
    g = torch.tensor([1.0, -0.5], device="cuda")
    _, lse = lib.linear_cross_entropy(h, w, y)
    dh, dw = lib.linear_cross_entropy_backward(h, w, y, lse, g)
    end_dh, end_dw = lib.linear_cross_entropy_backward(h, w[V - last:], y - (V - last), lse, g)
    finished()
    assert torch.equal(dw[V - last:], end_dw)
    h64, exact, mass = h.double(), 0.0, 0.0
    z = torch.cat([h64 @ w[v:v + 10_000].double().T for v in range(0, V, 10_000)], 1)
    dz = torch.softmax(z, 1)
    dz[torch.arange(T), y] -= 1
    dz *= g.double()[:, None]
    for v in range(0, V, 10_000):
        part = w[v:v + 10_000].double()
        exact = exact + dz[:, v:v + 10_000] @ part
        mass = mass + dz[:, v:v + 10_000].abs() @ part.abs()
    # a logit's 16384 products in sums of 2^8 steps: 2^-16 of sum |h w| (under 256), relative to dz; dH in
    # sums of under 2^11 steps; its rounding to bf16
    assert bool(((dh.double() - exact).abs() <= 2 ** -8 * exact.abs() + (2 ** -8 + 2 ** -13) * mass).all())


def test_both_losses_train_a_head():
    """The example: cross entropy and divergence fall together, and padding's NaN reaches no gradient."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_head.py")
    spec = importlib.util.spec_from_file_location("train_head", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    history = example.train(tokens=300, vocab=2000, depth=128, steps=12)
    finished()
    assert all(math.isfinite(v) for row in history for v in row)
    first, last = history[0], history[-1]
    assert last[0] < first[0] - 0.5 and last[1] < 0.7 * first[1]


def test_calls_from_several_threads():
    """Threads with streams and workspaces of their own get the bits a single call gives."""
    import threading
    lib = H.tg()
    cases = []
    for i, dtype in enumerate((BF16, F16, F32, BF16)):
        h, w, gen = head(130 + 40 * i, 900, 96, dtype, seed=i)
        y = targets_for(130 + 40 * i, 900, gen, 0.2)
        g = torch.rand(130 + 40 * i, device="cuda", generator=gen)
        cases.append((h, w, y, g, xent_both(h, w, y, g)))
    torch.cuda.synchronize()
    wrong = []

    def work(case):
        h, w, y, g, want = case
        stream = torch.cuda.Stream()
        for _ in range(5):
            loss, lse = lib.linear_cross_entropy(h, w, y, stream=stream.cuda_stream)
            dh, dw = lib.linear_cross_entropy_backward(h, w, y, lse, g, stream=stream.cuda_stream)
            stream.synchronize()
            for name, x in (("loss", loss), ("lse", lse), ("dh", dh), ("dw", dw)):
                if not torch.equal(x, want[name]):
                    wrong.append(name)

    threads = [threading.Thread(target=work, args=(c,)) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    finished()


@pytest.mark.parametrize("T", [3, 200], ids=["few_rows", "tiles"])
def test_captured_in_a_graph(T):
    """A step captured in a CUDA graph and replayed on new inputs gives the bits of plain calls."""
    V, D = 1500, 128
    h, w, gen = head(T, V, D, BF16, seed=1)
    y = targets_for(T, V, gen, 0.2)
    g = torch.rand(T, device="cuda", generator=gen)
    xent_both(h, w, y, g)  # first calls set kernel attributes and device records
    lib = H.tg()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, lse = lib.linear_cross_entropy(h, w, y)
        dh, dw = lib.linear_cross_entropy_backward(h, w, y, lse, g)
    for seed in (2, 3):
        h2, w2, gen = head(T, V, D, BF16, seed=seed)
        h.copy_(h2)
        w.copy_(w2)
        y.copy_(targets_for(T, V, gen, 0.3))
        graph.replay()
        want = xent_both(h, w, y, g)
        for name, x in (("loss", loss), ("lse", lse), ("dh", dh), ("dw", dw)):
            assert torch.equal(x, want[name]), name
