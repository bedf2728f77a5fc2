"""Views with overlapping rows: the expert-layer functions refuse the ones that a
leading dimension cannot describe, and take shared (expanded) experts and biases."""
import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from expert_helpers import check, grouped_ref, offsets_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def test_overlapping_rows_are_refused():
    x = torch.randn((6, 32), device="cuda").bfloat16()
    off = offsets_of([2, 4])
    row = torch.randn((2, 1, 16), device="cuda").bfloat16()
    col = torch.randn((2, 32, 1), device="cuda").bfloat16()
    flat = torch.randn(256, device="cuda").bfloat16()
    for w in (row.expand(2, 32, 16), col.expand(2, 32, 16), flat.as_strided((2, 32, 16), (64, 4, 1))):
        with pytest.raises(ValueError):
            G.grouped_matmul(x, w, off)
    with pytest.raises(ValueError):
        G.grouped_matmul(x[:1].expand(6, 32), torch.randn((2, 32, 16), device="cuda").bfloat16(), off)
    dy = torch.randn((6, 16), device="cuda").bfloat16()
    with pytest.raises(ValueError):
        G.grouped_weight_grad(x, dy, off, out=torch.zeros((2, 1, 16), device="cuda").expand(2, 32, 16))
    q, s, z = G.quantize_q4(torch.randn((16, 32), device="cuda"), 32, zero_points=True)
    for bad in ((q[:1].expand(16, 16), s, z), (q, s[:1].expand(16, 1), z), (q, s, z[:1].expand(16, 1))):
        with pytest.raises(ValueError):
            G.q4_matmul(x, bad[0], bad[1], 32, zeros=bad[2])


@pytest.mark.parametrize("K,N", [(40, 1), (1, 24), (33, 17)])
def test_shared_experts_and_one_wide_weights(K, N):
    gen = torch.Generator("cuda").manual_seed(0)
    x = torch.randn((50, K), device="cuda", generator=gen).bfloat16()
    off = offsets_of([20, 0, 30])
    w = torch.randn((3, K, N), device="cuda", generator=gen).bfloat16()
    b = torch.randn((1, N), device="cuda", generator=gen)
    for v in (w, w[:1].expand(3, K, N), w.transpose(1, 2).contiguous().transpose(1, 2)):
        ref, mag = grouped_ref(x, v, off, b.expand(3, N))
        check(G.grouped_matmul(x, v, off, bias=b.expand(3, N)), ref, mag, K, "bf16")
