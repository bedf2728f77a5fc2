"""What the operators around the products report of their launches: Plan.last_config() and the
log line of every call."""
import os
import subprocess
import sys

import pytest
import torch

import dense_gemm_epilogues_gb300 as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _data(T=300, E=40, d=128):
    gen = torch.Generator("cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, device="cuda", generator=gen).bfloat16()   # noqa: E731
    return rand(T, E), rand(T, d), rand(2 * T, d), rand(d, 256), rand(T, 256)


def _calls(plan):
    z, x, y, w, dy = _data()
    r = G.route(z, 2)
    return {"route": lambda: G.route(z, 2, plan=plan), "route_one": lambda: G.route(z[:9], 2, plan=plan),
            "route_grad": lambda: G.route_grad(z, r, dloss=1.0, plan=plan), "dispatch": lambda: G.dispatch(x, r, plan=plan),
            "combine": lambda: G.combine(y, r, plan=plan), "dispatch_grad": lambda: G.dispatch_grad(y, r, plan=plan),
            "combine_grad": lambda: G.combine_grad(x, y, r, plan=plan), "clip": lambda: G.clip_grad_norm([y], 1.0, plan=plan),
            "norm": lambda: G.grad_norm([x, y], plan=plan),
            "bias": lambda: G.linear_grad(dy, x, w, input_grad=False, weight_grad=False, plan=plan)}


@pytest.mark.parametrize("name", ["route", "route_one", "route_grad", "dispatch", "combine", "dispatch_grad", "combine_grad",
                                  "clip", "norm", "bias"])
def test_configuration_of_calls_without_a_product(name):
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    call = _calls(plan)[name]
    _, x, _, w, _ = _data()
    G.linear(x, w, plan=plan)
    assert plan.last_config()["kernel"] in (G.GEMM_KERNEL_TC, G.GEMM_KERNEL_TC_PAIR)
    call()
    c = plan.last_config()
    assert c["kernel"] == G.GEMM_KERNEL_SIMT and c["bm"] == c["bn"] == 0 and c["split_k"] == 1
    assert c["grid"] == 1 if name == "route_one" else c["grid"] > 1


def test_calls_that_launch_nothing():
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    z, x, y, w, dy = _data()
    r = G.route(z, 2)
    none = G.route(z[:0], 2)
    for call in (lambda: G.route_grad(z[:0], none, plan=plan), lambda: G.dispatch(x[:0], none, plan=plan),
                 lambda: G.dispatch(x[:, :0], r, plan=plan), lambda: G.combine(y[:0], none, plan=plan),
                 lambda: G.combine_grad(x[:0], y[:0], none, plan=plan)):
        G.linear(x, w, plan=plan)
        call()
        assert plan.last_config()["kernel"] == G.GEMM_KERNEL_NONE


def test_a_gradient_reports_its_last_product():
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    _, x, _, w, dy = _data()
    G.linear_grad(dy, x, w, plan=plan)
    assert plan.last_config()["kernel"] in (G.GEMM_KERNEL_TC, G.GEMM_KERNEL_TC_PAIR)


def test_log_lines():
    code = ("import torch, test_layers_reports as t; import dense_gemm_epilogues_gb300 as G; p = G.Plan(G.GEMM_BF16, G.GEMM_F32)\n"
            "for c in t._calls(p).values(): c()\ntorch.cuda.synchronize()")
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, GEMM_LOG="1", PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    run = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr
    names = [line.split()[1] for line in run.stderr.splitlines() if line.startswith("gemm: ")]
    for name, times in (("route", 3), ("route_grad", 1), ("dispatch", 1), ("combine", 2), ("combine_grad", 1), ("clip_norm", 2),
                        ("linear_grad", 1)):
        assert names.count(name) == times, (name, names)
