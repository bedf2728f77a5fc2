"""Values at the edges of the expert-layer operators' types: NaN under the fused ReLU."""
import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from expert_helpers import DT, U, check, grouped_ref, offsets_of, q4_weights, random_q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _same_with_nan(y, ref, mag, depth, out, extra=0.0):
    assert torch.equal(y.isnan(), ref.isnan())
    keep = ~ref.isnan()
    check(y[keep], ref[keep], mag[keep], depth, out, extra)


# Single CTAs and pairs; results negative and positive.
@pytest.mark.parametrize("counts,N", [([40, 0, 25], 300), ([600], 12000)], ids=str)
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_relu_of_grouped_products_keeps_nan(counts, N, out):
    gen, K, E = _gen(1), 72, len(counts)
    R, off = sum(counts), offsets_of(counts)
    x = torch.randn((R, K), device="cuda", generator=gen).bfloat16()
    w = torch.randn((E, K, N), device="cuda", generator=gen).bfloat16()
    b = torch.randn((E, N), device="cuda", generator=gen)
    x[7, 3], w[E - 1, 5, 11], b[0, 17] = (float("nan"),) * 3
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    y = G.grouped_matmul(x, w, off, bias=b, relu=True, out_dtype=DT[out], plan=plan)
    assert plan.device_status() == 0
    ref, mag = grouped_ref(x, w, off, b, True)
    assert ref[7].isnan().all() and ref[-1, 11].isnan() and ref[0, 17].isnan()
    _same_with_nan(y, ref, mag, K, out)


# A few rows, a prompt on single CTAs, a prompt on pairs.
@pytest.mark.parametrize("rows,N", [(5, 300), (300, 4096), (600, 12000)])
def test_relu_of_4_bit_products_keeps_nan(rows, N):
    gen, K = _gen(2), 256
    x = torch.randn((rows, K), device="cuda", generator=gen).bfloat16()
    q, s, z = random_q4(N, K, 64, DT["bf16"], True, gen)
    b = torch.randn(N, device="cuda", generator=gen)
    x[3, 9], s[20, 1], b[33] = (float("nan"),) * 3
    y = G.q4_matmul(x, q, s, 64, zeros=z, bias=b, relu=True, out_dtype=DT["f32"])
    w = q4_weights(q, s, z, K, 64)
    ref, mag = grouped_ref(x, w.mT[None], offsets_of([rows]), b, True)
    assert ref[3].isnan().all() and ref[:, 20].isnan().all() and ref[:, 33].isnan().all()
    _same_with_nan(y, ref, mag, K, "f32", U["bf16"] if rows > 32 else 0.0)
