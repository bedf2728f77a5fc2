"""Bounded waits of the expert-layer operators: a bound far below their run time makes the
waits expire; the kernels report GEMM_ERR_TIMEOUT, wind down and return, and the same plan
then gives the results it gave before."""
import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from expert_helpers import DT, offsets_of, random_q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


# On single CTAs and on pairs; 4-bit products inside and decoded once.
def _calls():
    gen = torch.Generator("cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, device="cuda", generator=gen).bfloat16()   # noqa: E731
    x, dy, w = rand(600, 2048), rand(600, 4096), rand(2, 2048, 4096)
    few, many = offsets_of([40, 24]), offsets_of([350, 250])
    q, s, z = random_q4(4096, 2048, 64, DT["bf16"], True, gen)
    g, stack = rand(300, 2000), rand(20, 400, 800)
    return {"grouped": lambda p: G.grouped_matmul(x[:64], w, few, plan=p),
            "grouped pairs": lambda p: G.grouped_matmul(x, w, many, plan=p),
            "gradient": lambda p: G.grouped_weight_grad(x[:64], dy[:64], few, plan=p),
            "gradient pairs": lambda p: G.grouped_weight_grad(x, dy, many, plan=p),
            "4-bit": lambda p: G.q4_matmul(x[:20], q, s, 64, zeros=z, plan=p),
            "4-bit once": lambda p: G.q4_matmul(x, q, s, 64, zeros=z, plan=p),
            "update": lambda p: G.orthogonalize(g, plan=p),
            "update pairs": lambda p: G.orthogonalize(stack, plan=p),
            "update f32": lambda p: G.orthogonalize(stack, out_dtype=DT["f32"], plan=p)}


@pytest.mark.parametrize("name", ["grouped", "grouped pairs", "gradient", "gradient pairs", "4-bit", "4-bit once",
                                  "update", "update pairs", "update f32"])
def test_bounded_waits_report_timeouts_and_the_plan_survives(name):
    call, plan = _calls()[name], G.Plan(G.GEMM_BF16, G.GEMM_F32)
    want = call(plan)
    assert plan.device_status() == 0
    G.gemm_plan_set_timeout(plan.handle, 200)       # 200 ns
    call(plan)
    # (a wait whose first try is granted does not expire: the hardware suspends it for a while)
    assert plan.device_status() in ((G.GEMM_ERR_TIMEOUT,) if name.startswith("update") else (0, G.GEMM_ERR_TIMEOUT))
    G.gemm_plan_set_timeout(plan.handle, 4_000_000_000)
    assert torch.equal(call(plan), want)
    assert plan.device_status() == 0
