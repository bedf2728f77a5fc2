"""Values at the edges of the expert-layer operators' types: NaN under the fused ReLU, and
4-bit weights whose scales lie outside fp16."""
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


# fp16 activations with scales of a wider type: weights below fp16's normal numbers, above its
# largest one, and of sizes that differ from column to column.  A weight is rounded once,
# relative to its column's largest scale (the groups of a column differ by at most 2^4 here),
# so the bound is that of a rounding to fp16.  Rows: inside the product; once, on single CTAs
# and on pairs.
@pytest.mark.parametrize("rows,N,experts", [(5, 300, 1), (300, 4096, 1), (600, 12000, 1), (300, 1000, 3)])
@pytest.mark.parametrize("sdt", ["f32", "bf16"])
@pytest.mark.parametrize("size", ["small", "large", "mixed"])
def test_4_bit_scales_outside_fp16(rows, N, experts, sdt, size):
    gen, K = _gen(3), 256
    x = torch.randn((rows, K), device="cuda", generator=gen).half()
    q, s, z = random_q4(N, K, 64, torch.float32, True, gen, experts)
    e = {"small": torch.full((N, 1), -28.0), "large": torch.full((N, 1), 24.0),
         "mixed": (torch.arange(N) * 7 % 80 - 40).float()[:, None]}[size].cuda()
    s = (s * torch.exp2(e)).to(DT[sdt])
    s[:, 4] = 0
    counts = [rows] if experts == 1 else [rows - 120, 0, 120]
    off = offsets_of(counts)
    plan = G.Plan(G.GEMM_F16, G.GEMM_F32)
    y = G.q4_matmul(x, q, s, 64, zeros=z, offsets=off, out_dtype=DT["f32"], plan=plan)
    assert plan.device_status() == 0
    w = q4_weights(q, s, z, K, 64)
    check(y, *grouped_ref(x, w.mT, off), K, "f32", U["f16"] if rows > 32 else 0.0)
