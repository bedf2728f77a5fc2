"""Bounded waits of fully connected layers: waits that run out are reported, and the plan gives
the same bits afterwards."""
import pytest
import torch

import dense_gemm_epilogues_gb300 as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _expire(M, K, N, layout, limit):
    """The plan's configuration after a call whose waits expire."""
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.randn((M, K), device="cuda", generator=gen).bfloat16()
    w = torch.randn((K, N) if layout == "kn" else (N, K), device="cuda", generator=gen).bfloat16()
    w = w if layout == "kn" else w.t()
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    want = G.linear(x, w, activation="gelu", plan=plan)
    assert plan.device_status() == 0
    G.gemm_plan_set_timeout(plan.handle, limit)
    G.linear(x, w, activation="gelu", plan=plan)
    assert plan.device_status() == G.GEMM_ERR_TIMEOUT
    G.gemm_plan_set_timeout(plan.handle, 4_000_000_000)
    assert torch.equal(G.linear(x, w, activation="gelu", plan=plan), want) and plan.device_status() == 0
    return plan.last_config()


# A limit below a microsecond gives a wait of the split kernel one look at its barrier: the
# hardware would hold a try for longer than these loads take.
@pytest.mark.parametrize("M,K,N", [(1, 4096, 11008), (5, 8192, 4096), (30, 8200, 1000), (64, 4096, 4096), (128, 4100, 11000)])
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_split_products(M, K, N, layout):
    assert _expire(M, K, N, layout, 1)["bk"] == 64


# The tile kernel's epilogue waits for a whole tile's products, 40 us and more.
@pytest.mark.parametrize("M,K,N,cta_group", [(384, 8192, 9984, 1), (2000, 32768, 6000, 2)])
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_tiles(M, K, N, cta_group, layout):
    c = _expire(M, K, N, layout, 200)
    assert c["bk"] == 128 and c["cta_group"] == cta_group
