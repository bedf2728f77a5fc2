"""Single-CTA stream-K: one plan for shapes of different tile widths and counts.  The
arrival counters must be zero for each launch, whatever partial sums the launches before
it left in the plan's scratch."""
import pytest
import torch

import dense_gemm_epilogues_gb300 as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _run(plan, M, N, K, seed):
    """A product of small integers: exact in fp32, in any order."""
    gen = torch.Generator("cuda").manual_seed(seed)
    a = torch.randint(-2, 3, (M, K), device="cuda", generator=gen).half()
    b = torch.randint(-2, 3, (K, N), device="cuda", generator=gen).half()
    d = torch.full((M, N), 7.5, device="cuda")
    G.matmul(a, b, out=d, plan=plan)
    assert plan.device_status() == 0 and plan.last_config()["sk_tiles"] > 0, plan.last_config()
    assert torch.equal(d.double(), a.double() @ b.double())
    return plan.last_config()["bn"]


@pytest.mark.parametrize("order", [(256, 128, 64), (64, 256, 128, 64), (128, 64, 256)])
def test_widths_in_turn(order, monkeypatch):
    monkeypatch.setenv("GEMM_TC_CTA_GROUP", "1")
    monkeypatch.setenv("GEMM_TC_SPLITK", "1")
    plan = G.Plan(G.GEMM_F16, G.GEMM_F32)
    for turn in range(2):
        for bn in order:
            monkeypatch.setenv("GEMM_TC_BN", str(bn))
            assert _run(plan, 384, 768, 4096, 10 * turn + bn) == bn


def test_shapes_in_turn_by_the_selector():
    plan = G.Plan(G.GEMM_F16, G.GEMM_F32)
    widths = [_run(plan, M, N, K, i) for i, (M, N, K) in
              enumerate([(128, 20000, 8192), (128, 512, 8192), (128, 10240, 16384), (128, 2048, 16384)])]
    assert widths == [256, 64, 128, 64]
