"""gemm_orthogonalize where a matrix lacks directions (the gradient of fewer rows than its
sizes) and for every output type.

What is rounded in a missing direction grows by a in every later step, and nothing in the
exact result is there to hide it, so these inputs show how precisely the operator holds X
between the products.  The bound is the error of the same steps with the roundings that
include/gemm.h states and exact products, times 1.3 for a bf16 result (the roundings are
the same in kind and number, but not bit by bit).  For fp16 and fp32 results the stated
roundings are those of fp32 arithmetic, and the sums' own order and truncation count as
well: four times the error of the plain fp32 steps, and 12 * 2^-23 for each of the
ceil(n / 16) additions that the longest sum makes (a common truncation of all sums moves
X X' by that much, which enters the result with (|b| + 2 |c|) / 0.7 = 12), and the
result's own rounding."""
import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from expert_helpers import DT, U, newton_schulz_ref

pytestmark = pytest.mark.gpu
A, B, C = 3.4445, -4.7750, 2.0315


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _matrix(m, n, rank, seed, batch=1):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn((batch, m, rank), device="cuda", generator=gen) @ \
        torch.randn((batch, rank, n), device="cuda", generator=gen)


def _half(x):
    return x.half().double()


def _stated_roundings(g, steps=5):
    """The steps with a bf16 result: X as a pair of fp16 numbers (times 1024), its first half
    in the products, E and F in fp16, a X by F's diagonal in the last two steps."""
    x = g.double() / (g.double().norm() + 1e-7) * 1024
    hi = _half(x)
    lo = _half(x - hi)
    eye = torch.eye(g.shape[0], device=g.device, dtype=torch.float64)
    for k in range(steps):
        h = 1.0 if k >= steps - 2 else 0.0
        a, b = A + B * h + C * h, B + 2 * C * h
        e = _half(hi @ hi.mT / 2 ** 20 - h * eye)
        f = _half(C * (e @ e.mT) + b * e + h * a * eye)
        x = f @ hi + (1 - h) * a * (hi + lo)
        hi = _half(x)
        lo = _half(x - hi)
    return x / 1024


def _plain(g, steps=5):
    x = g / (g.square().sum().sqrt() + 1e-7)
    for _ in range(steps):
        s = x @ x.mT
        x = A * x + (B * s + C * (s @ s)) @ x
    return x


def _rel(d, ref):
    return float((d.double() - ref).norm() / ref.norm())


# Single CTAs, pairs in a batch and alone.
@pytest.mark.parametrize("batch,m,n", [(1, 192, 256), (24, 200, 520), (1, 1100, 3000)])
@pytest.mark.parametrize("rank", [1, 4, 16, 97])
@pytest.mark.parametrize("tall", [False, True])
def test_few_rows(batch, m, n, rank, tall):
    g = _matrix(m, n, rank, 1, batch)
    gt = g.mT.contiguous() if tall else g
    plan = G.Plan(G.GEMM_F32, G.GEMM_F32)
    for out in ("bf16", "f16", "f32"):
        d = G.orthogonalize(gt, out_dtype=DT[out], plan=plan)
        assert plan.device_status() == 0
        d = d.mT if tall else d
        for z in {0, batch // 2, batch - 1}:
            ref = newton_schulz_ref(g[z])
            if out == "bf16":
                bound = 1.3 * _rel(_stated_roundings(g[z]).bfloat16(), ref)
            else:
                bound = 4 * _rel(_plain(g[z]), ref) + 12 * -(-n // 16) * 2.0 ** -23 + U[out]
            assert _rel(d[z], ref) <= bound, (out, z, _rel(d[z], ref), bound)


@pytest.mark.parametrize("m,n", [(1, 2), (1, 300), (2, 5), (3, 8), (5, 21), (16, 64), (16, 17)])
@pytest.mark.parametrize("tall", [False, True])
def test_matrices_of_a_few_rows(m, n, tall):
    """300 matrices of a few singular values, where no rounding averages out: a bf16 result
    is as near as its own rounding and fp32 steps allow."""
    gen = torch.Generator("cuda").manual_seed(3)
    g = torch.randn((300, m, n), device="cuda", generator=gen)
    plan = G.Plan(G.GEMM_F32, G.GEMM_F32)
    d = G.orthogonalize(g.mT.contiguous() if tall else g, plan=plan)
    assert plan.device_status() == 0
    d = d.mT if tall else d
    for z in range(300):
        ref = newton_schulz_ref(g[z])
        bound = U["bf16"] + 4 * _rel(_plain(g[z]), ref) + 12 * -(-n // 16) * 2.0 ** -23
        assert _rel(d[z], ref) <= bound, (z, _rel(d[z], ref), bound)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n", [(1, 1), (40, 1), (7, 9), (333, 1001), (257, 255), (1536, 520)])
def test_wide_results_are_as_precise_as_their_type(m, n, dtype):
    """Full-rank matrices, fp16 and fp32 results of every input type."""
    gen = torch.Generator("cuda").manual_seed(2)
    g = (0.01 * torch.randn((m, n), device="cuda", generator=gen)).to(DT[dtype])
    wide = g if m <= n else g.mT
    ref = newton_schulz_ref(wide)
    plan = G.Plan(G.DTYPE_CODES[dtype], G.GEMM_F32)
    for out in ("f16", "f32"):
        d = G.orthogonalize(g, out_dtype=DT[out], plan=plan)
        assert plan.device_status() == 0
        d = d if m <= n else d.mT
        bound = 4 * _rel(_plain(wide.float()), ref) + 12 * -(-max(m, n) // 16) * 2.0 ** -23 + U[out]
        assert _rel(d, ref) <= bound, (out, _rel(d, ref), bound)
