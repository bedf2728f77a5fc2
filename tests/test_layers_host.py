"""Host-side checks of the operators around the products (no GPU needed): the bindings' structs
are the header's, null plans are refused, and the Python functions refuse what they can tell
from shapes, types and views before they touch a device."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import dense_gemm_epilogues_gb300 as G

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = ["gemm_linear_t", "gemm_routing_t", "gemm_tensor_t"]


@pytest.fixture(scope="module", autouse=True)
def lib():
    from dense_gemm_epilogues_gb300 import build
    build.build()
    return G.load_library()


def test_structs_match_the_header(tmp_path):
    fields = [(s, n) for s in STRUCTS for n, _ in getattr(G, s)._fields_]
    lines = "".join(f'printf("%zu\\n", offsetof({s}, {n}));' for s, n in fields)
    lines += "".join(f'printf("%zu\\n", sizeof({s}));' for s in STRUCTS)
    src = tmp_path / "t.c"
    src.write_text(f'#include <stddef.h>\n#include <stdio.h>\n#include "gemm.h"\nint main(void) {{ {lines} return 0; }}\n')
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    want = [getattr(getattr(G, s), n).offset for s, n in fields] + [ctypes.sizeof(getattr(G, s)) for s in STRUCTS]
    assert got == want


def test_activation_codes_match_the_header():
    text = open(os.path.join(ROOT, "include", "gemm.h")).read()
    for name in ("NONE", "RELU", "GELU", "GELU_TANH", "SILU"):
        assert f"GEMM_LINEAR_{name} = {getattr(G, 'GEMM_LINEAR_' + name)}" in text


def test_null_plans_are_refused(lib):
    r = G.gemm_routing_t()
    assert lib.gemm_route(None, 1, 1, None, 1, None, r, None) == G.GEMM_ERR_INVALID_ARG
    assert lib.gemm_route_grad(None, 1, 1, None, 1, r, None, 1.0, None, None, 1, None) == G.GEMM_ERR_INVALID_ARG
    assert lib.gemm_dispatch(None, 1, 1, 1, 1, None, 1, None, None, None, 1, None) == G.GEMM_ERR_INVALID_ARG
    assert lib.gemm_combine(None, 1, 1, 1, 1, None, 1, None, None, None, 1, None, 1, None) == G.GEMM_ERR_INVALID_ARG
    assert lib.gemm_combine_grad(None, 1, 1, 1, 1, None, 1, None, 1, None, None, None, None, 1, None, None) == G.GEMM_ERR_INVALID_ARG
    assert lib.gemm_clip_norm(None, 0, None, 1.0, 0.0, None, None) == G.GEMM_ERR_INVALID_ARG
    assert lib.gemm_run_linear(None, 1, 1, 1, 1, None, 1, None, 1, None, 1, None, None) == G.GEMM_ERR_INVALID_ARG
    assert lib.gemm_run_linear_grad(None, 1, 1, 1, 1, None, 1, None, 1, 0, None, 1, None, 1, None, 1, None, 1, 0, None,
                                    None) == G.GEMM_ERR_INVALID_ARG


def _routing(tokens=4, experts=8, top=2, **kw):
    f = dict(weights=torch.zeros((tokens, top)), experts=torch.zeros((tokens, top), dtype=torch.int32),
             slots=torch.zeros((tokens, top), dtype=torch.int32), counts=torch.zeros(experts, dtype=torch.int32),
             offsets=torch.zeros(experts + 1, dtype=torch.int32), routed=torch.zeros((), dtype=torch.int32))
    f.update(kw)
    return G.Routing(**f)


def test_refusals_without_a_device():
    z, x, y = torch.zeros((4, 8)), torch.zeros((4, 16)).half(), torch.zeros((8, 16)).half()
    w = torch.zeros((16, 32)).half()
    a = torch.zeros(100)
    r = _routing()
    for bad in (lambda: G.route(z, 0), lambda: G.route(z, 9), lambda: G.route(z.t(), 2), lambda: G.route(z, 2),
                lambda: G.route(z, 2, mask=torch.zeros(5, dtype=torch.bool)), lambda: G.route(z, 2, mask=torch.zeros(4)),
                lambda: G.route_grad(z[:3], r), lambda: G.route_grad(z, _routing(weights=torch.zeros((4, 2)).double())),
                lambda: G.route_grad(z, _routing(counts=torch.zeros(7, dtype=torch.int32))),
                lambda: G.route_grad(z, r, dweights=torch.zeros((4, 3))), lambda: G.route_grad(z, r, out=z.half()),
                lambda: G.route_grad(z, r, dloss=torch.zeros(2)),
                lambda: G.dispatch(x[:3], r), lambda: G.dispatch(x, r), lambda: G.dispatch(x, r, out=y[:, :8]),
                lambda: G.dispatch(x, _routing(slots=torch.zeros((4, 2)))), lambda: G.dispatch(x, _routing(offsets=torch.zeros(9))),
                lambda: G.combine(y, r, residual=x.float()), lambda: G.combine(y, _routing(weights=torch.zeros((2, 4)))),
                lambda: G.combine_grad(x[:, :8], y, r), lambda: G.combine_grad(x.float(), y, r),
                lambda: G.linear(x, w[:8]), lambda: G.linear(x, w.float()), lambda: G.linear(x, w, activation="tanh"),
                lambda: G.linear(x, w), lambda: G.linear(x, w.expand(16, 32)[:, ::2]),
                lambda: G.linear_grad(x, x, w), lambda: G.linear_grad(torch.zeros((4, 32)).half(), x, w, activation="gelu"),
                lambda: G.linear_grad(torch.zeros((4, 32)), x, w),
                lambda: G.TensorList([a, a]), lambda: G.TensorList([a[:60], a[50:]]), lambda: G.TensorList([a[::2]]),
                lambda: G.TensorList([a], out=[]), lambda: G.TensorList([a], out=[a[:99]]),
                lambda: G.TensorList([a[:50]], out=[a[10:60]]), lambda: G.TensorList([a.double()]),
                lambda: G.TensorList([a]), lambda: G.clip_grad_norm([a], 1.0)):
        with pytest.raises(ValueError):
            bad()


def test_bounds_of_clipping():
    for max_norm, eps in ((-1.0, 0.0), (math.nan, 0.0), (1.0, -1.0), (1.0, math.nan), (1.0, math.inf)):
        with pytest.raises(ValueError):
            G.clip_grad_norm([], max_norm, eps=eps)
