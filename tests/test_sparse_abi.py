"""The C ABI of a sparse layer's operators and of the gradients' norm on the host:
declared and exported names, struct layouts, sizes and refusals.  No call here
reaches the GPU."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# fake, well-separated device addresses: nothing dereferences them
A0, B0, C0, D0, E0, F0, G0, H0 = (0x1000000000 * (i + 1) for i in range(8))


@pytest.fixture(scope="module")
def tg():
    from tests.conftest import build_library
    build_library()
    import tiled_dense_gemm_02_gb300 as tg
    return tg


def header(name):
    return open(os.path.join(ROOT, "include", name)).read()


def test_headers_and_exports_agree(tg):
    for name, exports in (("tgemm_experts.h", tg.EXPERT_EXPORTS), ("tgemm_grads.h", tg.GRAD_EXPORTS)):
        names = set(re.findall(r"^\s*TGEMM_API\s+int\s+(tgemm_\w+)\s*\(", header(name), re.M))
        assert names == set(exports)
        for n in names:
            assert hasattr(tg.library(), n)
    for name, value in re.findall(r"#define\s+TGEMM_(ROUTE_MAX_\w+|GRAD_MAX_\w+)\s+(\d+)",
                                  header("tgemm_experts.h") + header("tgemm_grads.h")):
        assert getattr(tg, name) == int(value)
    for name, value in re.findall(r"TGEMM_(ROUTE_(?:SOFTMAX|SIGMOID|GROUP_\w+)) = (\d)", header("tgemm_experts.h")):
        assert getattr(tg, name) == int(value)


def fields(text, struct):
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (struct, struct), text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    return [" ".join(d.split()) for d in body.split(";") if d.strip()]


def test_option_structs_match_the_header(tg):
    decls = fields(header("tgemm_experts.h"), "tgemm_route_options")
    assert decls == ["int scoring", "int renormalize", "float scale", "int groups", "int top_groups", "int group_score",
                     "int reserved[2]"]
    assert [f for f, _ in tg.RouteOptions._fields_] == [d.split()[1].split("[")[0] for d in decls]
    assert ctypes.sizeof(tg.RouteOptions) == 32


def route(tg, T=64, E=32, k=4, x=A0, ld=32, dtype=2, bias=B0, ids=C0, w=D0, **o):
    return tg.route_forward(T, E, k, x, ld, dtype, bias, ids, w, o or None)


def unroute(tg, T=64, E=32, k=4, x=A0, ld=32, dtype=2, ids=C0, g=D0, out=E0, ld_out=32, **o):
    return tg.route_backward(T, E, k, x, ld, dtype, ids, g, out, ld_out, o or None)


def test_route_refusals(tg):
    bad = tg.ERR_INVALID_VALUE
    for call in (route, unroute):
        for args in ({"T": -1}, {"E": 0}, {"k": 0}, {"k": 33}, {"ld": 31}, {"x": 0}, {"ids": 0}, {"scoring": 2},
                     {"scoring": -1}, {"renormalize": 2}, {"scale": -1.0}, {"scale": float("inf")},
                     {"scale": float("nan")}, {"groups": 3}, {"groups": -1}, {"groups": 2, "top_groups": 3},
                     {"top_groups": 2}, {"groups": 16, "top_groups": 1}, {"group_score": 2}, {"top_groups": -1}):
            assert call(tg, **args) == bad, args
        assert call(tg, dtype=3) == call(tg, dtype=9) == tg.ERR_UNSUPPORTED_DTYPE
        assert call(tg, x=A0 + 1) == call(tg, dtype=0, x=A0 + 2) == call(tg, ids=C0 + 4) == tg.ERR_MISALIGNED
        assert call(tg, E=1025, ld=1025, ld_out=1025) if call is unroute else call(tg, E=1025, ld=1025) == tg.ERR_TOO_LARGE
        assert call(tg, T=1 << 31) == call(tg, ld=1 << 31) == tg.ERR_TOO_LARGE
        assert call(tg, E=64, ld=64, groups=64, **({"ld_out": 64} if call is unroute else {})) == tg.ERR_TOO_LARGE
        assert call(tg, T=0, x=0) == tg.OK
    assert route(tg, E=64, ld=64, k=33) == unroute(tg, E=64, ld=64, ld_out=64, k=33) == tg.ERR_TOO_LARGE
    assert route(tg, w=0) == unroute(tg, g=0) == unroute(tg, out=0) == unroute(tg, ld_out=31) == bad
    assert route(tg, w=D0 + 2) == route(tg, bias=B0 + 1) == unroute(tg, g=D0 + 2) == unroute(tg, out=E0 + 1) == tg.ERR_MISALIGNED
    for args in ({"ids": A0}, {"w": A0 + 64}, {"bias": C0}, {"w": C0 + 8}, {"bias": D0 + 1020}):
        assert route(tg, **args) == tg.ERR_ALIAS, args
    for args in ({"out": A0}, {"out": C0}, {"out": D0}, {"out": A0 + 64 * 32 * 2 - 2}):
        assert unroute(tg, **args) == tg.ERR_ALIAS, args


def test_reserved_route_options_must_be_zero(tg):
    o = tg.RouteOptions()
    o.reserved[1] = 1
    assert tg.route_forward(4, 8, 2, A0, 8, 0, 0, B0, C0, o) == tg.ERR_INVALID_VALUE


def clip(tg, grads=(A0, B0), counts=(100, 200), dtypes=(0, 2), outputs=None, limit=1.0, norm=C0, ws=D0, n=1 << 20):
    return tg.grad_clip(grads, counts, dtypes, outputs, limit, norm, ws, n)


def test_gradient_refusals(tg):
    bad = tg.ERR_INVALID_VALUE
    for args in ({"counts": (-1, 5)}, {"grads": (0, B0)}, {"outputs": (0, B0)}, {"limit": -0.5}, {"limit": float("nan")},
                 {"norm": 0}, {"ws": 0}, {"ws": D0 + 128}, {"n": 4863}):
        assert clip(tg, **args) == bad, args
    assert clip(tg, dtypes=(0, 3)) == clip(tg, dtypes=(0, -1)) == tg.ERR_UNSUPPORTED_DTYPE
    assert clip(tg, grads=(A0 + 2, B0)) == clip(tg, grads=(A0, B0 + 1)) == clip(tg, norm=C0 + 2) == \
        clip(tg, outputs=(A0, B0 + 1)) == tg.ERR_MISALIGNED
    assert clip(tg, counts=(1 << 40, 5)) == tg.ERR_TOO_LARGE
    alias = tg.ERR_ALIAS
    assert clip(tg, grads=(A0, A0)) == clip(tg, grads=(A0, A0 + 396)) == clip(tg, norm=A0) == clip(tg, ws=B0) == alias
    assert clip(tg, outputs=(A0 + 4, B0)) == clip(tg, outputs=(E0, E0 + 396)) == clip(tg, outputs=(B0, F0)) == alias
    assert clip(tg, outputs=(C0, F0)) == clip(tg, outputs=(F0, D0 + 512)) == alias
    assert tg.grad_norm((A0, B0), (100, 200), (0, 9), C0, D0, 1 << 20) == tg.ERR_UNSUPPORTED_DTYPE
    assert tg.grad_norm((A0, B0), (100, 200), (0, 2), A0, D0, 1 << 20) == alias


def test_gradient_workspace(tg):
    assert tg.grad_workspace_size(0) == tg.grad_workspace_size(1000) == (tg.OK, 4864)
    assert tg.grad_workspace_size(1001) == (tg.OK, 2 * 4864)
    assert tg.grad_workspace_size(-1)[0] == tg.ERR_INVALID_VALUE
    assert tg.grad_workspace_size(1 << 21)[0] == tg.ERR_TOO_LARGE
    assert tg.library().tgemm_grad_workspace_size(4, None) == tg.ERR_INVALID_VALUE


def test_headers_are_c(tmp_path):
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("gcc not found")
    src = tmp_path / "both.c"
    src.write_text('#include "tgemm_experts.h"\n#include "tgemm_grads.h"\n#include <stdio.h>\n'
                   'int main(void) { printf("%zu\\n", sizeof(tgemm_route_options)); return 0; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(tmp_path / "both")], check=True)
    assert subprocess.run([str(tmp_path / "both")], capture_output=True, text=True, check=True).stdout == "32\n"


def forward(tg, T=64, E=4, k=2, D=32, F=48, x=A0, ldx=32, w_in=B0, ld_in=32, w_out=C0, ld_out=48, ids=D0, w=E0, dtype=2, out=F0,
            ldo=32, saved=0, sn=0, ws=G0, n=1 << 24, **o):
    return tg.experts_forward(T, E, k, D, F, x, ldx, w_in, ld_in, w_out, ld_out, ids, w, dtype, out, ldo, saved, sn, o or None, ws, n)


DX0, DI0, DO0, DW0 = (0x1000000000 * (i + 20) for i in range(4))


def backward(tg, T=64, E=4, k=2, D=32, F=48, x=A0, ldx=32, w_in=B0, ld_in=32, w_out=C0, ld_out=48, w=E0, dtype=2, saved=H0, sn=1 << 24,
             g=F0, ldg=32, dx=DX0, lddx=32, di=DI0, ldi=32, do=DO0, ldo=48, dw=DW0, ws=G0, n=1 << 24, **o):
    return tg.experts_backward(T, E, k, D, F, x, ldx, w_in, ld_in, w_out, ld_out, w, saved, sn, g, ldg, dtype, dx, lddx, di, ldi, do,
                               ldo, dw, o or None, ws, n)


def test_expert_refusals(tg):
    bad = tg.ERR_INVALID_VALUE
    for call in (forward, backward):
        for args in ({"T": -1}, {"E": 0}, {"k": 0}, {"D": 0}, {"F": 0}, {"ldx": 31}, {"ld_in": 31}, {"ld_out": 47}, {"x": 0}, {"w_in": 0},
                     {"w_out": 0}, {"w": 0}, {"ws": 0}, {"ws": G0 + 128}, {"n": 1000}, {"wait_timeout_us": -1}):
            assert call(tg, **args) == bad, args
        assert call(tg, dtype=0) == call(tg, dtype=3) == tg.ERR_UNSUPPORTED_DTYPE
        assert call(tg, x=A0 + 1) == call(tg, w_in=B0 + 1) == call(tg, w_out=C0 + 1) == call(tg, w=E0 + 2) == tg.ERR_MISALIGNED
        big = tg.ERR_TOO_LARGE
        assert call(tg, E=1025) == call(tg, k=1 << 16) == call(tg, D=1 << 24, ldx=1 << 24, ld_in=1 << 24) == big
        assert call(tg, T=1 << 30, k=2) == call(tg, ldx=1 << 31) == call(tg, E=1024, F=1 << 21, ld_out=1 << 21) == big
    assert forward(tg, ids=0) == forward(tg, out=0) == forward(tg, ldo=31) == forward(tg, saved=H0, sn=100) == bad
    assert forward(tg, saved=H0 + 64, sn=1 << 24) == bad
    assert backward(tg, saved=0) == backward(tg, sn=100) == backward(tg, g=0) == backward(tg, ldg=31) == bad
    assert backward(tg, lddx=31) == backward(tg, ldi=31) == backward(tg, ldo=47) == bad
    assert forward(tg, ids=D0 + 4) == forward(tg, out=F0 + 1) == backward(tg, dw=DW0 + 2) == backward(tg, g=F0 + 1) == tg.ERR_MISALIGNED
    for args in ({"out": A0}, {"out": B0 + 64}, {"ws": A0}, {"out": E0}, {"saved": G0, "sn": 1 << 24}, {"out": G0}, {"ids": F0}):
        assert forward(tg, **args) == tg.ERR_ALIAS, args
    for args in ({"dx": A0}, {"di": B0}, {"do": C0 + 2}, {"dw": E0}, {"dx": DI0}, {"do": DI0 + 4 * 96 * 32 * 2 - 2}, {"ws": H0}, {"dx": H0},
                 {"g": DX0}):
        assert backward(tg, **args) == tg.ERR_ALIAS, args
    assert forward(tg, T=0, x=0, ids=0, out=0, ws=0) == tg.OK
    assert backward(tg, dx=0, di=0, do=0, dw=0) == tg.OK
    o = tg.ExpertsOptions()
    o.reserved[2] = 1
    assert tg.experts_forward(4, 2, 1, 8, 8, A0, 8, B0, 8, C0, 8, D0, E0, 2, F0, 8, 0, 0, o, G0, 1 << 20) == bad


def test_expert_sizes(tg):
    import itertools
    decls = fields(header("tgemm_experts.h"), "tgemm_experts_options")
    assert decls == ["int wait_timeout_us", "int reserved[3]"] and ctypes.sizeof(tg.ExpertsOptions) == 16
    for T, E, k, D, F in itertools.product((1, 7, 300), (1, 5, 300), (1, 4), (8, 100), (8, 70)):
        rows = -(-(T * k + 31 * min(E, T * k)) // 32) * 32
        st, saved = tg.experts_saved_size(T, E, k, D, F, 2)
        assert st == tg.OK and saved >= rows * (8 * F + 2 * D)
        for backward in (0, 1):
            st, n = tg.experts_workspace_size(backward, T, E, k, D, F, 0, D, 0, F, 2)
            assert st == tg.OK and n >= rows * (2 * F + 2 * D + (4 * F if backward else 0))
            # misaligned weights are copied
            copies = (E * 2 * F * D * 2 if D % 8 == 0 else 0) + (E * D * F * 2 if F % 8 == 0 else 0)
            # (an empty part takes 256 bytes)
            assert tg.experts_workspace_size(backward, T, E, k, D, F, 2, D, 2, F, 2)[1] >= n + copies - 512
            assert tg.experts_workspace_size(backward, T, E, k, D, F, 0, D, 0, F, 1)[1] > n  # fp16's rows to join are fp32
    assert tg.experts_workspace_size(2, 4, 2, 1, 8, 8, 0, 8, 0, 8, 2)[0] == tg.ERR_INVALID_VALUE
    assert tg.experts_workspace_size(0, 4, 2, 1, 8, 8, 0, 7, 0, 8, 2)[0] == tg.ERR_INVALID_VALUE
    assert tg.experts_workspace_size(0, 4, 2, 1, 8, 8, 0, 8, 0, 8, 0)[0] == tg.ERR_UNSUPPORTED_DTYPE
    assert tg.experts_saved_size(0, 2, 1, 8, 8, 2) == tg.experts_workspace_size(1, 0, 2, 1, 8, 8, 0, 8, 0, 8, 2) == (tg.OK, 0)
