"""gemm_orthogonalize against the Newton-Schulz steps in 64 bits: wide, tall and
square, odd sizes, batches, every type, layouts and padding, zero and non-finite
matrices, other coefficients and step counts.

Bound: X and the two small products of a step are rounded to fp16 (2^-11).  In
the last step, where every singular value is near one, a rounding of the small
products enters with |b| + 2|c| and X itself with |a|, over a + b + c = 0.7, so
one step adds at most about (2.7 + 2 * 2.0 + 3.4) / 0.7 * 2^-11 of the result's
norm if all of it lined up; the roundings are independent, and a tenth of that
per step over five steps, 0.5 * 14 * 2^-11 = 3.5e-3, bounds the Frobenius error.
The output's own rounding adds its unit.  (Singular values far below the others
are resolved less well: the inputs here have a spread as in the table below.)"""
import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from expert_helpers import DT, U, newton_schulz_ref

pytestmark = pytest.mark.gpu
BOUND = 3.5e-3


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _matrix(batch, m, n, dtype, seed, strong=4.0):
    """Noise with a few directions `strong` times above its largest singular value."""
    gen = torch.Generator("cuda").manual_seed(seed)
    r = min(4, m, n)
    g = torch.randn((batch, m, n), device="cuda", generator=gen)
    u = torch.randn((batch, m, r), device="cuda", generator=gen)
    v = torch.randn((batch, r, n), device="cuda", generator=gen)
    return (0.01 * (g + strong * (m ** 0.5 + n ** 0.5) / (m * n) ** 0.5 * (u @ v))).to(DT[dtype])


def _check(got, g, out, **kw):
    ref = newton_schulz_ref(g, **kw)
    for a, r in zip(got.double().reshape(-1, *g.shape[-2:]), ref.reshape(-1, *g.shape[-2:])):
        assert (a - r).norm() <= (BOUND + U[out]) * r.norm(), float((a - r).norm() / r.norm())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("batch,m,n", [(1, 64, 64), (1, 128, 256), (3, 256, 128), (1, 1, 1), (2, 1, 40), (1, 40, 1),
                                       (1, 7, 9), (2, 333, 1001), (1, 1001, 333), (1, 256, 256), (1, 257, 255),
                                       (5, 130, 384), (1, 512, 2048), (1, 1536, 520), (2, 640, 640)])
def test_orthogonalize(batch, m, n, dtype):
    g = _matrix(batch, m, n, dtype, 1)
    plan = G.Plan(G.DTYPE_CODES[dtype], G.GEMM_F32)
    for out in ("f32", "bf16"):
        d = G.orthogonalize(g, out_dtype=DT[out], plan=plan)
        assert d.dtype == DT[out] and plan.device_status() == 0
        _check(d, g, out)


@pytest.mark.parametrize("m,n", [(200, 320), (320, 200)])
def test_two_dimensions_layouts_and_guard_bands(m, n):
    g = _matrix(1, m, n, "f32", 2)[0]
    ref = G.orthogonalize(g, out_dtype=DT["f32"])
    _check(ref, g, "f32")
    col = g.t().contiguous().t()                         # column-major
    d = G.orthogonalize(col, out_dtype=DT["f32"])
    assert torch.equal(d, ref)
    wide = torch.full((m + 2, n + 13), float("nan"), device="cuda")
    wide[1:-1, 5:5 + n] = g
    buf = torch.full((m + 2, n + 9), 4.0, device="cuda", dtype=DT["bf16"])
    G.orthogonalize(wide[1:-1, 5:5 + n], out=buf[1:-1, 3:3 + n])
    _check(buf[1:-1, 3:3 + n].contiguous(), g, "bf16")
    buf[1:-1, 3:3 + n] = 4
    assert (buf == 4).all()
    keep = g.clone()
    G.orthogonalize(g)
    assert torch.equal(g, keep)                          # the input is only read


def test_shared_input_and_transpose():
    g = _matrix(1, 96, 160, "bf16", 3)
    d = G.orthogonalize(g.expand(3, 96, 160), out=torch.empty((3, 96, 160), device="cuda"))
    assert torch.equal(d[0], d[1]) and torch.equal(d[0], d[2])
    t = G.orthogonalize(g[0].t(), out=torch.empty((96, 160), device="cuda").t())
    assert torch.equal(t.t(), d[0])


@pytest.mark.parametrize("scale", [1e-12, 1e-3, 1.0, 1e12])
def test_scale_of_the_input_does_not_matter(scale):
    g = _matrix(1, 150, 200, "f32", 4)[0]
    d = G.orthogonalize(g * scale, eps=0.0, out_dtype=DT["f32"])
    _check(d, g * scale, "f32", eps=0.0)


def test_zero_and_non_finite_matrices():
    g = _matrix(4, 72, 100, "f32", 5)
    g[1] = 0
    g[2, 3, 4] = float("nan")
    g[3, 70, 99] = float("inf")
    d = G.orthogonalize(g, out_dtype=DT["f32"])
    assert (d[1] == 0).all() and d[2].isnan().all() and d[3].isnan().all()
    _check(d[0], g[0], "f32")


@pytest.mark.parametrize("steps,coeffs", [(0, (1.0, 0.0, 0.0)), (1, (3.4445, -4.7750, 2.0315)), (2, (1.5, -0.5, 0.0)),
                                          (12, (1.875, -1.25, 0.375))])
def test_steps_and_coefficients(steps, coeffs):
    g = _matrix(1, 120, 130, "f32", 6)[0]
    d = G.orthogonalize(g, steps=steps, coeffs=coeffs, out_dtype=DT["f32"])
    _check(d, g, "f32", steps=steps, coeffs=coeffs)


def test_result_is_nearly_orthonormal():
    g = _matrix(1, 300, 700, "bf16", 7, strong=1.0)[0]
    d = G.orthogonalize(g, out_dtype=DT["f32"]).double()
    s = torch.linalg.svdvals(d)
    assert 0.6 < float(s.min()) and float(s.max()) < 1.3


def test_repeated_calls_agree_bit_for_bit():
    g = _matrix(2, 500, 900, "bf16", 8)
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    d = G.orthogonalize(g, plan=plan)
    for _ in range(3):
        assert torch.equal(d, G.orthogonalize(g, plan=plan))


def test_empty_and_refusals():
    assert G.orthogonalize(torch.zeros((0, 4, 4), device="cuda")).shape == (0, 4, 4)
    assert G.orthogonalize(torch.zeros((2, 0, 4), device="cuda")).shape == (2, 0, 4)
    g = torch.ones((8, 12), device="cuda")
    for bad in (lambda: G.orthogonalize(g[0]), lambda: G.orthogonalize(g, out=torch.zeros((12, 8), device="cuda")),
                lambda: G.orthogonalize(torch.ones((8, 24), device="cuda")[:, ::2]),
                lambda: G.orthogonalize(g, out=torch.zeros((8, 12)))):
        with pytest.raises(ValueError):
            bad()
    plan = G.Plan(G.GEMM_F32, G.GEMM_F32)

    def code(batch=1, M=8, N=12, steps=5, coeffs=(1.0, 1.0, 1.0), eps=1e-7, ldg=12, ldd=12, sd=96, out=G.GEMM_F32,
             G_=g.data_ptr(), h=plan.handle):
        with pytest.raises(G.GemmError) as e:
            G.gemm_orthogonalize(h, batch, M, N, steps, coeffs, eps, G_, ldg, 96, g.data_ptr(), ldd, sd, out)
        return e.value.status

    for kw in (dict(batch=-1), dict(M=-1), dict(steps=-1), dict(steps=65), dict(eps=-1.0), dict(eps=float("nan")),
               dict(coeffs=(1.0, float("inf"), 1.0)), dict(ldg=11), dict(ldd=11), dict(batch=2, sd=90), dict(G_=None),
               dict(out=G.GEMM_S8), dict(h=None)):
        assert code(**kw) == G.GEMM_ERR_INVALID_ARG, kw
    p8 = G.Plan(G.GEMM_S8, G.GEMM_S32)
    assert code(h=p8.handle) == G.GEMM_ERR_UNSUPPORTED
