"""Offsets of grouped products at their limits: the most groups that a call takes, and bad
offsets that give the same rows to many groups."""
import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from expert_helpers import DT, check, grouped_ref, offsets_of, wgrad_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


@pytest.mark.parametrize("groups", [31, 33, 1000, 1024])
def test_many_groups(groups):
    gen = torch.Generator("cuda").manual_seed(1)
    counts = [(7 * g) % 5 + (140 if g % 97 == 5 else 0) for g in range(groups)]
    off, R = offsets_of(counts), sum(counts)
    x = torch.randn((R, 64), device="cuda", generator=gen).bfloat16()
    dy = torch.randn((R, 136), device="cuda", generator=gen).bfloat16()
    w = torch.randn((groups, 64, 136), device="cuda", generator=gen).bfloat16()
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    y = G.grouped_matmul(x, w, off, out_dtype=DT["f32"], plan=plan)
    dw = G.grouped_weight_grad(x, dy, off, out_dtype=DT["f32"], plan=plan)
    assert plan.device_status() == 0
    check(y, *grouped_ref(x, w, off), 64, "f32")
    check(dw, *wgrad_ref(x, dy, off), max(counts), "f32")


@pytest.mark.parametrize("groups", [40, 1024])
def test_rows_of_many_groups_stay_inside_the_buffer(groups):
    """Offsets 0, R, 0, R, ...: every other group has all rows.  Reported, and nothing
    outside the buffer is written."""
    R, N = 500, 264
    gen = torch.Generator("cuda").manual_seed(2)
    x = torch.randn((R, 64), device="cuda", generator=gen).bfloat16()
    w = torch.randn((groups, 64, N), device="cuda", generator=gen).bfloat16()
    off = torch.tensor([R * (g % 2) for g in range(groups + 1)], dtype=torch.int32, device="cuda")
    buf = torch.full((R + 8, N), 5.0, device="cuda", dtype=DT["bf16"])
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    G.grouped_matmul(x, w, off, out=buf[4:-4], plan=plan)
    assert plan.device_status() == G.GEMM_ERR_INVALID_ARG
    assert (buf[:4] == 5).all() and (buf[-4:] == 5).all() and not (buf[4:-4] == 5).all(1).any()
