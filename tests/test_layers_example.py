"""What the example of an expert layer adds up, and the gradients that it takes back, against
64-bit forms: outputs are kept in fp32, a row's gradient is rounded once.

A sum of two fp32 products is off by at most 4 2^-23 of the sum of their absolute values; a
gradient by two fp32 roundings and half a step of bf16."""
import os
import sys

import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from layer_helpers import EPS, U, within

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("tokens", [1, 300])
def test_sums_and_gradients_of_the_example(tokens):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import expert_layer
    gen = torch.Generator("cuda").manual_seed(1)
    d = 64
    r = G.route(torch.randn((tokens, 8), device="cuda", generator=gen), expert_layer.TOP)
    y = torch.randn((tokens * expert_layer.TOP, d), device="cuda", generator=gen).bfloat16()
    dout = torch.randn((tokens, d), device="cuda", generator=gen) * 1e-3
    plan = G.Plan(G.GEMM_F32, G.GEMM_F32)
    slots, w = r.slots.long(), r.weights.double()
    rows = w[..., None] * y.double()[slots]
    out = expert_layer.added(y, r, plan)
    assert out.dtype is torch.float32
    within(out, rows.sum(1), 4 * EPS * rows.abs().sum(1))
    dy = expert_layer.row_gradients(dout, y, r, plan)
    assert dy.dtype is torch.bfloat16
    ref = torch.empty_like(y, dtype=torch.float64)
    ref[slots.flatten()] = (w[..., None] * dout.double()[:, None, :]).reshape(-1, d)
    within(dy, ref, (U["bf16"] * (1 + 2.0 ** -22) + 2.0 ** -23) * ref.abs())
    assert plan.device_status() == 0
