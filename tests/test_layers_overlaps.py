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
