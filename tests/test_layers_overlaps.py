"""Outputs that are an input, where the formula reads what it would overwrite: refused."""
import pytest
import torch

import dense_gemm_epilogues_gb300 as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _refused(call):
    with pytest.raises(G.GemmError) as e:
        call()
    assert e.value.status == G.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_in_place(dtype):
    """With one expert per token the sorted rows have the tokens' shape."""
    gen = torch.Generator("cuda").manual_seed(1)
    x, y, dout = (torch.randn((40, 64), device="cuda", generator=gen).to(dtype) for _ in range(3))
    r = G.route(torch.randn((40, 8), device="cuda", generator=gen), 1)
    kept = [t.clone() for t in (x, y, dout)]
    _refused(lambda: G.dispatch(x, r, out=x))
    _refused(lambda: G.combine(y, r, out=y))
    _refused(lambda: G.combine(y, r, residual=x, out=y))
    _refused(lambda: G.dispatch_grad(y, r, out=y))
    _refused(lambda: G.combine_grad(dout, y, r, out=y))
    _refused(lambda: G.combine_grad(dout, y, r, out=dout))
    assert all(torch.equal(a, b) for a, b in zip((x, y, dout), kept))
    want = G.combine(y, r, residual=x)
    assert torch.equal(G.combine(y, r, residual=x, out=x), want)   # (a token's own row is read before it is written)


def test_rows_of_nothing():
    r = G.route(torch.zeros((4, 8), device="cuda"), 1)
    e = torch.empty((4, 0), device="cuda")
    assert G.dispatch(e, r, out=e) is e and G.combine(e, r, out=e) is e and G.combine_grad(e, e, r, out=e)[0] is e


@pytest.mark.parametrize("M", [8, 600])
def test_layers_in_place(M):
    gen = torch.Generator("cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, device="cuda", generator=gen).bfloat16()   # noqa: E731
    x, w, res = rand(M, 128), rand(128, 128), rand(M, 128)
    kept = [t.clone() for t in (x, w, res)]
    _refused(lambda: G.linear(x, w, out=x))
    _refused(lambda: G.linear(x, w, residual=res, out=x))
    _refused(lambda: G.linear(rand(128, 128), w, out=w))
    plan, lib = G.Plan(G.GEMM_BF16, G.GEMM_F32), G.load_library()
    D = torch.empty_like(res)
    for pre in (x, w, res, D):
        e = G.gemm_linear_t(None, G.GEMM_F32, G.GEMM_LINEAR_GELU, res.data_ptr(), 128, pre.data_ptr(), 128, G.GEMM_BF16)
        assert lib.gemm_run_linear(plan.handle, G.GEMM_OP_T, M, 128, 128, x.data_ptr(), 128, w.data_ptr(), 128,
                                   D.data_ptr(), 128, e, None) == G.GEMM_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((x, w, res), kept))
    want = G.linear(x, w, activation="gelu", residual=res)
    assert torch.equal(G.linear(x, w, activation="gelu", residual=res, out=res), want)


@pytest.mark.parametrize("act", [G.GEMM_LINEAR_NONE, G.GEMM_LINEAR_SILU])
def test_gradients_in_place(act):
    gen = torch.Generator("cuda").manual_seed(1)
    dy, pre, x, w, dx, dw = (torch.randn((128, 128), device="cuda", generator=gen).bfloat16() for _ in range(6))
    db = torch.empty(128, device="cuda")
    plan, lib = G.Plan(G.GEMM_BF16, G.GEMM_F32), G.load_library()

    def status(dx=dx, dw=dw, db=db):
        return lib.gemm_run_linear_grad(plan.handle, G.GEMM_OP_T, 128, 128, 128, dy.data_ptr(), 128, pre.data_ptr(), 128, act,
                                        x.data_ptr(), 128, w.data_ptr(), 128, dx.data_ptr(), 128, dw.data_ptr(), 128,
                                        G.GEMM_BF16, db.data_ptr(), torch.cuda.current_stream().cuda_stream)

    for t in (dy, x, w) + ((pre,) if act else ()):
        for name in ("dx", "dw", "db"):
            assert status(**{name: t}) == G.GEMM_ERR_INVALID_ARG
    assert status() == G.GEMM_OK
    if not act:   # (not read without an activation: its memory may be used)
        assert status(dx=pre) == G.GEMM_OK and torch.equal(pre, dx)
