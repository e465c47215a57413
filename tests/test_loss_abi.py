"""The vocabulary-head losses' C ABI on the host: declared and exported names,
struct layout, workspace sizes and refusals.  No call here reaches the GPU."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tgemm_loss.h")

# fake, well-separated device addresses: nothing dereferences them
H0, W0, Y0, L0, S0, G0, DH0, DW0, WS0, T0 = (0x1000000000 * (i + 1) for i in range(10))


@pytest.fixture(scope="module")
def tg():
    from tests.conftest import build_library
    build_library()
    import tiled_dense_gemm_02_gb300 as tg
    return tg


def test_header_and_exports_agree(tg):
    text = open(HEADER).read()
    names = set(re.findall(r"^\s*TGEMM_API\s+int\s+(tgemm_\w+)\s*\(", text, re.M))
    assert names == set(tg.LOSS_EXPORTS)
    for name in names:
        assert hasattr(tg.library(), name)
    assert int(re.search(r"#define\s+TGEMM_DISTILL_MAX_K\s+(\d+)", text).group(1)) == tg.DISTILL_MAX_K


def test_options_struct_matches_header(tg):
    body = re.search(r"typedef struct tgemm_loss_options \{(.*?)\} tgemm_loss_options;", open(HEADER).read(), re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    decls = [" ".join(d.split()) for d in body.split(";") if d.strip()]
    assert decls == ["float scale", "float label_smoothing", "float z_loss", "int piece", "int64_t ignore_index",
                     "int wait_timeout_us", "int reserved[3]"]
    assert [f for f, _ in tg.LossOptions._fields_] == [d.split()[1].split("[")[0] for d in decls]
    assert ctypes.sizeof(tg.LossOptions) == 40 and tg.LossOptions.ignore_index.offset == 16


def xent_f(tg, T=64, V=300, D=64, H=H0, ldh=64, W=W0, ldw=64, y=Y0, dtype=2, loss=L0, lse=S0, ws=WS0, n=1 << 30, **o):
    options = tg.LossOptions(ignore_index=-100, **o)
    return tg.xent_forward(T, V, D, H, ldh, W, ldw, y, dtype, loss, lse, options, ws, n)


def xent_b(tg, T=64, V=300, D=64, H=H0, ldh=64, W=W0, ldw=64, y=Y0, lse=S0, g=G0, dtype=2, dh=DH0, lddh=64, dw=DW0,
           lddw=64, ws=WS0, n=1 << 30, **o):
    options = tg.LossOptions(ignore_index=-100, **o)
    return tg.xent_backward(T, V, D, H, ldh, W, ldw, y, lse, g, dtype, dh, lddh, dw, lddw, options, ws, n)


def distill_f(tg, T=64, V=300, D=64, K=8, ids=Y0, ld_ids=8, t=T0, ld_t=8, dtype=2, loss=L0, lse=S0, ws=WS0, n=1 << 30,
              **o):
    options = tg.LossOptions(**o)
    return tg.distill_forward(T, V, D, K, H0, 64, W0, 64, ids, ld_ids, t, ld_t, dtype, loss, lse, options, ws, n)


def distill_b(tg, T=64, V=300, D=64, K=8, ids=Y0, ld_ids=8, t=T0, ld_t=8, lse=S0, g=G0, dtype=2, dh=DH0, lddh=64,
              dw=DW0, lddw=64, ws=WS0, n=1 << 30, **o):
    options = tg.LossOptions(**o)
    return tg.distill_backward(T, V, D, K, H0, 64, W0, 64, ids, ld_ids, t, ld_t, lse, g, dtype, dh, lddh, dw, lddw,
                               options, ws, n)


@pytest.mark.parametrize("bad", [
    {"T": -1}, {"V": 0}, {"V": -4}, {"D": 0}, {"ldh": 63}, {"ldw": 63}, {"H": 0}, {"W": 0}, {"y": 0}, {"loss": 0},
    {"lse": 0}, {"ws": 0}, {"ws": WS0 + 8}, {"n": 1000}, {"scale": -1.0}, {"scale": float("nan")},
    {"scale": float("inf")}, {"label_smoothing": -0.1}, {"label_smoothing": 1.5}, {"label_smoothing": float("nan")},
    {"z_loss": -1.0}, {"z_loss": float("inf")}, {"piece": -256}, {"piece": 100}, {"wait_timeout_us": -1},
    {"reserved": (ctypes.c_int * 3)(0, 1, 0)},
])
def test_forward_refuses_invalid_values(tg, bad):
    assert xent_f(tg, **bad) == tg.ERR_INVALID_VALUE


@pytest.mark.parametrize("bad", [
    {"T": -1}, {"V": 0}, {"D": 0}, {"ldh": 1}, {"ldw": 1}, {"lddh": 63}, {"lddw": 63}, {"H": 0}, {"W": 0}, {"y": 0},
    {"lse": 0}, {"g": 0}, {"ws": 0}, {"ws": WS0 + 128}, {"n": 1000}, {"piece": 1},
])
def test_backward_refuses_invalid_values(tg, bad):
    assert xent_b(tg, **bad) == tg.ERR_INVALID_VALUE


@pytest.mark.parametrize("bad", [
    {"K": 0}, {"K": -1}, {"ld_ids": 7}, {"ld_t": 7}, {"ids": 0}, {"t": 0}, {"label_smoothing": 0.1}, {"z_loss": 0.1},
    {"ws": 0}, {"n": 1000},
])
def test_distillation_refuses_invalid_values(tg, bad):
    assert distill_f(tg, **bad) == tg.ERR_INVALID_VALUE
    assert distill_b(tg, **bad) == tg.ERR_INVALID_VALUE


def test_other_refusals(tg):
    for dtype in (-1, 3, 4, 9):  # a 16-bit input with fp32 output is no form of these losses
        assert xent_f(tg, dtype=dtype) == tg.ERR_UNSUPPORTED_DTYPE
        assert distill_b(tg, dtype=dtype) == tg.ERR_UNSUPPORTED_DTYPE
    assert xent_f(tg, H=H0 + 1) == tg.ERR_MISALIGNED
    assert xent_f(tg, W=W0 + 2, dtype=0) == tg.ERR_MISALIGNED
    assert xent_f(tg, y=Y0 + 4) == tg.ERR_MISALIGNED
    assert xent_f(tg, loss=L0 + 2) == tg.ERR_MISALIGNED
    assert xent_b(tg, g=G0 + 1) == tg.ERR_MISALIGNED
    assert xent_b(tg, dw=DW0 + 1) == tg.ERR_MISALIGNED
    assert distill_f(tg, t=T0 + 2) == tg.ERR_MISALIGNED
    assert xent_f(tg, loss=S0) == tg.ERR_ALIAS
    assert xent_f(tg, lse=H0 + 64) == tg.ERR_ALIAS
    assert xent_f(tg, ws=W0) == tg.ERR_ALIAS
    assert xent_b(tg, dh=H0) == tg.ERR_ALIAS
    assert xent_b(tg, dw=W0 + 128) == tg.ERR_ALIAS
    assert xent_b(tg, dw=DH0 + 64) == tg.ERR_ALIAS
    assert xent_b(tg, dh=G0) == tg.ERR_ALIAS
    assert distill_f(tg, loss=T0) == tg.ERR_ALIAS
    big = 1 << 31
    assert xent_f(tg, T=big) == tg.ERR_TOO_LARGE
    assert xent_f(tg, V=big) == tg.ERR_TOO_LARGE
    assert xent_f(tg, D=big, ldh=big, ldw=big) == tg.ERR_TOO_LARGE
    assert xent_f(tg, ldh=big) == tg.ERR_TOO_LARGE
    assert distill_f(tg, K=257, ld_ids=257, ld_t=257) == tg.ERR_TOO_LARGE


def test_nothing_to_do_is_no_error(tg):
    assert xent_f(tg, T=0, H=0, W=0, y=0, loss=0, lse=0, ws=0, n=0) == tg.OK
    assert distill_f(tg, T=0, ids=0, t=0, loss=0, lse=0, ws=0, n=0) == tg.OK
    assert xent_b(tg, dh=0, dw=0, ws=0, n=0) == tg.OK


def test_workspace_sizes(tg):
    def size(backward, T, V, D, K=0, W=W0, ldw=None, dtype=2, **o):
        st, n = tg.loss_workspace_size(backward, T, V, D, K, W, D if ldw is None else ldw, dtype, o or None)
        assert st == tg.OK
        return n
    assert size(False, 0, 300, 64) == 0
    # nothing of the size of the logits, however large the vocabulary
    T, V, D = 8192, 131072, 4096
    assert size(False, T, V, D) < T * D * 2 + T * V // 16
    assert size(True, T, V, D) < T * V // 2
    # a smaller piece of the gradient takes less
    assert size(True, T, V, D, piece=4096) < size(True, T, V, D)
    # rows off the 16-byte grid add a piece of W
    assert size(False, 64, 5000, 100, ldw=101) > size(False, 64, 5000, 100, ldw=104) + 5000 * 100 * 2
    assert size(True, 64, 5000, 100, W=W0 + 2, ldw=104) > size(True, 64, 5000, 100, ldw=104)
    assert size(False, 64, 5000, 64, K=256) > size(False, 64, 5000, 64, K=1)
    for args in ((2, 64, 300, 64, 0, W0, 64, 2), (0, 64, 300, 64, -1, W0, 64, 2), (0, -1, 300, 64, 0, W0, 64, 2),
                 (0, 64, 300, 64, 0, W0, 63, 2)):
        assert tg.loss_workspace_size(*args)[0] == tg.ERR_INVALID_VALUE
    assert tg.loss_workspace_size(0, 64, 300, 64, 257, W0, 64, 2)[0] == tg.ERR_TOO_LARGE
    assert tg.library().tgemm_loss_workspace_size(0, 64, 300, 64, 0, W0, 64, 2, None, None) == tg.ERR_INVALID_VALUE


def test_tensor_functions_refuse_bad_arguments(tg):
    import torch
    h, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(10, 8, dtype=torch.bfloat16)
    y = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: tg.linear_cross_entropy(h, w, y),                              # not on a CUDA device
                 lambda: tg.linear_cross_entropy(h, w.float(), y),
                 lambda: tg.linear_cross_entropy(h, torch.zeros(10, 9, dtype=torch.bfloat16), y),
                 lambda: tg.linear_cross_entropy(h[0], w, y),
                 lambda: tg.linear_cross_entropy(h.double(), w.double(), y),
                 lambda: tg.linear_cross_entropy(h, w, y, scale=0.0),
                 lambda: tg.linear_cross_entropy(torch.zeros(8, 4, dtype=torch.bfloat16).t(), w, y),
                 lambda: tg.linear_cross_entropy(h[:1].expand(4, 8), w, y),
                 lambda: tg.linear_distillation(h, w, torch.zeros(4, 3, dtype=torch.int64), torch.zeros(4, 3),
                                                temperature=0.0)):
        with pytest.raises(ValueError):
            call()


def test_header_from_c(tg, tmp_path):
    """The header compiles as C, and a C caller sees the binding's struct layout and the same sizes and refusals."""
    import subprocess
    src = tmp_path / "caller.c"
    src.write_text(r'''
#include <stddef.h>
#include <stdio.h>
#include "tgemm_loss.h"
int main(void) {
  tgemm_loss_options o = {0};
  size_t n = 0;
  o.ignore_index = -100;
  printf("%zu %zu %zu ", sizeof o, offsetof(tgemm_loss_options, ignore_index), offsetof(tgemm_loss_options, reserved));
  printf("%d ", tgemm_loss_workspace_size(1, 64, 5000, 100, 0, (const void*)0x1000, 101, TGEMM_BF16, &o, &n));
  printf("%zu ", n);
  printf("%d\n", tgemm_xent_forward(-1, 10, 10, 0, 10, 0, 10, 0, TGEMM_BF16, &o, 0, 0, 0, 0, 0));
  return 0;
}
''')
    exe = tmp_path / "caller"
    lib = os.path.join(ROOT, "tiled_dense_gemm_02_gb300")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe),
                    os.path.join(lib, "libtgemm.so"), f"-Wl,-rpath,{lib}"], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    st, n = tg.loss_workspace_size(True, 64, 5000, 100, 0, 0x1000, 101, tg.BF16)
    assert st == tg.OK
    assert [int(v) for v in got] == [ctypes.sizeof(tg.LossOptions), tg.LossOptions.ignore_index.offset,
                                     tg.LossOptions.reserved.offset, tg.OK, n, tg.ERR_INVALID_VALUE]
