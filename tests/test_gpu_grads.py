"""The norm over many gradients and their clipping on the GPU, against 64 bits.

The norm: squares are added in fp32 at most 32 at a time (each addition off by
2^-24 of a sum of positive terms) and from there in 64 bits, the root is rounded to
fp32: within 33 * 2^-24 / 2 + 2^-24 of the exact one.  The factor inherits the root's 16.5 * 2^-24 and
its own rounding; a scaled value is off by that, the product's rounding and half
a step of its type."""
import math

import pytest
import torch

from tests import gpu_harness as H

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    H.tg()
    torch.cuda.set_device(0)


def exact_norm(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))


def check_norm(got, grads):
    want = exact_norm(grads)
    assert got.shape == () and got.dtype == F32
    assert abs(float(got) - want) <= 18 * U * want, (float(got), want)
    return want


def check_scaled(out, grads, norm, max_norm):
    f = max_norm / norm if norm > max_norm else 1.0
    for o, g in zip(out, grads):
        if f == 1.0:
            assert torch.equal(o, g)
            continue
        want = f * g.double()
        step = {BF16: 0.0, F16: 2.0 ** -25, F32: 2.0 ** -150}[g.dtype]
        bound = want.abs() * (20 * U + torch.finfo(g.dtype).eps / 2) + step
        assert o.dtype == g.dtype and bool(((o.double() - want).abs() <= bound).all())


def some(sizes, dtypes, seed=0, spread=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(spread * (1 + i % 5) * torch.randn(n, device="cuda", generator=gen)).to(dtypes[i % len(dtypes)])
            for i, n in enumerate(sizes)]


LISTS = {"one_value": [1], "small": [1, 2, 3, 7, 8, 9, 15, 16, 17], "a_chunk": [8192, 8191, 8193, 4096, 4097],
         "empty_among": [0, 5, 0, 3000, 0], "forty": [101] * 40, "forty_one": [101 + i for i in range(41)],
         "thousand": [(37 * i) % 500 for i in range(1000)], "more": [(29 * i) % 300 + 1 for i in range(2100)],
         "large": [3_000_001, 64, 1_000_003]}


@pytest.mark.parametrize("dtypes", [(F32,), (BF16,), (F16,), (BF16, F32, F16)], ids=["f32", "bf16", "f16", "mixed"])
@pytest.mark.parametrize("name", LISTS)
def test_norm_and_clipping(name, dtypes):
    lib = H.tg()
    grads = some(LISTS[name], dtypes, seed=len(name))
    norm = check_norm(lib.gradient_norm(grads), grads)
    for limit in (0.25 * norm, 4.0 * norm, 0.0, math.inf):
        limit = float(torch.tensor(limit, dtype=F32))
        out = [torch.full_like(g, 77.0) for g in grads]
        check_norm(lib.clip_gradients(grads, limit, outputs=out), grads)
        check_scaled(out, grads, norm, limit)
        mine = [g.clone() for g in grads]
        check_norm(lib.clip_gradients(mine, limit), grads)
        for a, b in zip(mine, out):
            assert torch.equal(a, b)


def test_tensors_off_every_boundary_and_their_neighbours():
    """Gradients that share one buffer: nothing between or beside them changes; outputs at other offsets."""
    lib = H.tg()
    for dtype in (BF16, F16, F32):
        flat = torch.randn(40_000, device="cuda").to(dtype)
        spans, at = [], 3
        for i in range(60):
            n = (i * 97) % 613 + 1
            spans.append((at, at + n))
            at += n + i % 3
        grads = [flat[a:b] for a, b in spans]
        norm = exact_norm(grads)
        other = torch.full((41_000,), 7.0, device="cuda", dtype=dtype)
        out = [other[a + 5:b + 5] for a, b in spans]
        lib.clip_gradients(grads, norm / 3, outputs=out)
        check_scaled(out, grads, norm, norm / 3)
        hit = torch.zeros(41_000, dtype=torch.bool, device="cuda")
        for a, b in spans:
            hit[a + 5:b + 5] = True
        assert bool((other[~hit] == 7.0).all())
        before = flat.clone()
        lib.clip_gradients(grads, norm / 3)
        assert torch.equal(flat[~hit[5:40_005]], before[~hit[5:40_005]])
        check_scaled(grads, [before[a:b] for a, b in spans], norm, norm / 3)


@pytest.mark.parametrize("dtype,values", [(F32, (1e30, 3e38)), (F32, (1e-30, 1e-44)), (BF16, (2e38, 1e-38)), (F16, (65504.0, 6e-8)),
                                          (F32, (1e30, 1e-30)), (F32, (0.0, 0.0))])
def test_values_whose_squares_leave_fp32(dtype, values):
    lib = H.tg()
    grads = [torch.full((5000,), values[0], device="cuda").to(dtype), torch.full((3001,), values[1], device="cuda").to(dtype)]
    want = exact_norm(grads)
    got = float(lib.gradient_norm(grads))
    if want > torch.finfo(F32).max:
        assert got == math.inf
        return
    assert abs(got - want) <= 18 * U * want + 2.0 ** -150
    if 1e-20 < want:
        out = [torch.empty_like(g) for g in grads]
        limit = float(torch.tensor(want / 8, dtype=F32))
        lib.clip_gradients(grads, limit, outputs=out)
        check_scaled(out, grads, want, limit)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_norm_that_is_no_number_scales_nothing(bad):
    lib = H.tg()
    grads = some([1000, 333], (BF16, F32))
    grads[1][77] = bad
    kept = [g.clone() for g in grads]
    got = float(lib.clip_gradients(grads, 0.1))
    assert math.isnan(got) if math.isnan(bad) else got == math.inf
    for a, b in zip(grads, kept):
        assert torch.equal(a.view(torch.int16 if a.dtype == BF16 else torch.int32), b.view(torch.int16 if b.dtype == BF16 else torch.int32))


def test_dense_layouts_and_refusals():
    lib = H.tg()
    t = torch.randn(30, 40, device="cuda").t()
    last = torch.randn(2, 3, 4, 5, device="cuda").contiguous(memory_format=torch.channels_last)
    check_norm(lib.gradient_norm([t, last]), [t, last])
    out = torch.empty(30, 40, device="cuda").t()
    norm = exact_norm([t])
    lib.clip_gradients([t], norm / 2, outputs=[out])
    check_scaled([out], [t], norm, float(torch.tensor(norm / 2, dtype=F32)))
    wide = torch.randn(30, 40, device="cuda")
    for call in (lambda: lib.gradient_norm([wide[:, :20]]), lambda: lib.gradient_norm([wide.expand(2, 30, 40)]),
                 lambda: lib.gradient_norm([]), lambda: lib.gradient_norm([wide, wide.cpu()]),
                 lambda: lib.gradient_norm([wide.double()]), lambda: lib.clip_gradients([wide], -1.0),
                 lambda: lib.clip_gradients([wide], math.nan), lambda: lib.clip_gradients([wide], 1.0, outputs=[]),
                 lambda: lib.clip_gradients([wide], 1.0, outputs=[wide.bfloat16()]),
                 lambda: lib.clip_gradients([wide], 1.0, outputs=[torch.empty(40, 30, device="cuda").t()])):
        with pytest.raises(ValueError):
            call()
    for grads, outputs in (([wide, wide], None), ([wide, wide[3:5]], None), ([wide[:20], wide[20:]], [wide[1:21], torch.empty(10, 40, device="cuda")])):
        with pytest.raises(lib.TgemmError) as e:
            lib.clip_gradients(grads, 1.0, outputs=outputs)
        assert e.value.status == lib.ERR_ALIAS
    check_norm(lib.gradient_norm([wide, wide]), [wide, wide])  # nothing is written: the same tensor may count twice


def test_same_bits_every_time_in_a_graph_and_on_another_stream():
    lib = H.tg()
    grads = some([5_000_000, 123, 77_777], (BF16, F32))
    out = [torch.empty_like(g) for g in grads]

    def step():
        return lib.clip_gradients(grads, 1.0, outputs=out)

    want = float(step())
    first = [o.clone() for o in out]
    for _ in range(3):
        assert float(step()) == want
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = lib.clip_gradients(grads, 1.0, outputs=out, stream=side.cuda_stream)
    side.synchronize()
    assert float(got) == want and all(torch.equal(a, b) for a, b in zip(out, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = step()
    for seed in (5, 6):
        for g, new in zip(grads, some([5_000_000, 123, 77_777], (BF16, F32), seed=seed)):
            g.copy_(new)
        graph.replay()
        got = float(norm), [o.clone() for o in out]
        assert got[0] == float(step()) and all(torch.equal(a, b) for a, b in zip(out, got[1]))
