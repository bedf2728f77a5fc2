"""Rows between tokens and experts (dispatch, combine and their gradients) against 64-bit forms.

Copies are compared for equality.  A sum of n fp32 products is off by (n + 1) 2^-23 of the
sum of their absolute values at most, and half a step of its type."""
import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from layer_helpers import DT, EPS, TINY, U, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _routing(tokens, experts, top, seed=0, padded=True):
    z = torch.randn((tokens, experts), device="cuda", generator=_gen(seed))
    if tokens > 2 and experts > top:
        z[1, top - 1:] = -float("inf")       # a token with fewer experts
    return G.route(z, top, mask=torch.arange(tokens, device="cuda") % 6 != 5 if padded else None)


def _rand(shape, dtype, seed, odd=False):
    """odd: rows at an odd pitch and address, NaN around them."""
    v = torch.randn(shape, device="cuda", generator=_gen(seed)).to(DT[dtype])
    if not odd:
        return v
    wide = torch.full((shape[0], shape[1] + 5), float("nan"), device="cuda", dtype=DT[dtype])
    wide[:, 3:3 + shape[1]] = v
    return wide[:, 3:3 + shape[1]]


SIZES = [(1, 4, 1, 8), (1, 4, 4, 1), (7, 8, 2, 64), (16, 8, 2, 1024), (33, 5, 5, 129), (100, 16, 3, 264), (65, 40, 9, 1000),
         (50, 64, 32, 40), (3000, 64, 6, 16), (5000, 8, 2, 72)]


@pytest.mark.parametrize("tokens,experts,top,width", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("odd", [False, True])
def test_exchange(tokens, experts, top, width, dtype, odd):
    r = _routing(tokens, experts, top)
    R = tokens * top
    x, y = _rand((tokens, width), dtype, 1, odd), _rand((R, width), dtype, 2, odd)
    res, dout = _rand((tokens, width), dtype, 3, odd), _rand((tokens, width), dtype, 4, odd)
    slots, used = r.slots.long(), r.slots >= 0
    t_of = torch.arange(tokens, device="cuda")[:, None].expand(-1, top)
    # dispatch, into a buffer of its own and into the caller's
    sent = torch.zeros((R, width), device="cuda", dtype=DT[dtype])
    sent[slots[used]] = x[t_of[used]]
    assert torch.equal(G.dispatch(x, r), sent)
    out = _rand((R, width), dtype, 5, odd)
    assert G.dispatch(x, r, out=out) is out and torch.equal(out, sent)
    # combine
    w = torch.where(used, r.weights, 0.0).double()
    rows = torch.where(used[..., None], y.double()[slots.clamp(min=0)], 0.0)
    for residual in (None, res):
        ref = (w[..., None] * rows).sum(1) + (residual.double() if residual is not None else 0.0)
        mag = (w[..., None] * rows.abs()).sum(1) + (residual.double().abs() if residual is not None else 0.0)
        tol = U[dtype] * ref.abs() + (top + 2) * EPS * mag + TINY[dtype]
        within(G.combine(y, r, residual=residual), ref, tol, "combine")
    # dispatch_grad: weights of one
    ref, mag = rows.sum(1), rows.abs().sum(1)
    within(G.dispatch_grad(y, r), ref, U[dtype] * ref.abs() + (top + 2) * EPS * mag + TINY[dtype], "dispatch_grad")
    # combine_grad
    dy, dw = G.combine_grad(dout, y, r)
    ref = torch.zeros((R, width), device="cuda", dtype=torch.float64)
    ref[slots[used]] = (w[..., None] * dout.double()[:, None, :])[used]
    within(dy, ref, U[dtype] * ref.abs() * (1 + 1e-6) + 2.0 ** -24 * ref.abs() + TINY[dtype], "dy")
    ref = (rows * dout.double()[:, None, :]).sum(-1)
    mag = (rows * dout.double()[:, None, :]).abs().sum(-1)
    within(dw, ref, (width + 1) * 2.0 ** -24 * mag, "dweights")
    assert (dw[~used] == 0).all()
    assert G.default_plan_status() == 0


def test_residual_in_place_and_rows_that_are_not_read():
    r = _routing(200, 16, 4)
    y, res = _rand((800, 96), "bf16", 1), _rand((200, 96), "bf16", 2)
    y[int(r.offsets[-1]):] = float("nan")
    want = G.combine(y, r, residual=res)
    assert not want.isnan().any()
    assert G.combine(y, r, residual=res, out=res) is res and torch.equal(res, want)
    dy, dw = G.combine_grad(res, y, r)
    assert not dy.isnan().any() and not dw.isnan().any()


@pytest.mark.parametrize("width", [64, 61])
def test_nothing_is_written_around_the_outputs(width):
    T, top = 90, 3
    r = _routing(T, 16, top)
    x, y = _rand((T, width), "bf16", 1), _rand((T * top, width), "bf16", 2)
    for call, rows in ((lambda o: G.dispatch(x, r, out=o), T * top), (lambda o: G.combine(y, r, residual=x, out=o), T),
                       (lambda o: G.dispatch_grad(y, r, out=o), T), (lambda o: G.combine_grad(x, y, r, out=o), T * top)):
        wide = torch.full((rows + 4, width + 24), 7.0, device="cuda", dtype=torch.bfloat16)
        call(wide[2:-2, 8:8 + width])
        inner = torch.zeros_like(wide, dtype=torch.bool)
        inner[2:-2, 8:8 + width] = True
        assert (wide[~inner] == 7).all() and not (wide[inner] == 7).all()


def test_bad_slots_touch_nothing_and_are_reported():
    r = _routing(40, 8, 2, padded=False)
    bad = r.slots.clone()
    bad[3, 1], bad[9, 0], bad[11, 0] = 80, 2 ** 31 - 1, -7
    r = r._replace(slots=bad)
    x = _rand((40, 64), "f16", 1)
    plan = G.Plan(G.GEMM_F16, G.GEMM_F32)
    buf = torch.zeros((90, 64), device="cuda", dtype=torch.float16)
    for call in (lambda: G.dispatch(x, r, out=buf[:80], plan=plan), lambda: G.combine(buf[:80], r, plan=plan),
                 lambda: G.combine_grad(x, buf[:80], r, plan=plan)):
        call()
        assert plan.device_status() == G.GEMM_ERR_INVALID_ARG
        assert plan.device_status() == 0
    assert (buf[80:] == 0).all()
    dw = G.combine_grad(x, torch.ones((80, 64), device="cuda", dtype=torch.float16), r, plan=plan)[1]
    assert dw[3, 1] == 0 and dw[9, 0] == 0 and dw[11, 0] == 0
    plan.device_status()


def test_a_buffer_past_four_gigabytes():
    """Byte offsets past 32 bits: the last rows of a buffer of 5 GB."""
    tokens, top, width = 40000, 2, 32768
    slots = torch.arange(tokens * top, device="cuda", dtype=torch.int32).view(tokens, top)
    off = torch.tensor([0, tokens * top], dtype=torch.int32, device="cuda")
    r = G.Routing(torch.full((tokens, top), 0.5, device="cuda"), torch.zeros_like(slots), slots, off[1:], off,
                  off[:1].view(()))
    x = torch.randn((tokens, width), device="cuda", generator=_gen(1)).bfloat16()
    sent = G.dispatch(x, r)
    assert torch.equal(sent[-6:], x[-3:].repeat_interleave(2, 0)) and torch.equal(sent[:6], x[:3].repeat_interleave(2, 0))
    assert torch.equal(sent.view(tokens, top, width)[:, 1], x)
    assert torch.equal(G.combine(sent, r), x)
    del sent


def test_graph_stream_and_run_together():
    """route, dispatch, grouped products, combine and their gradients as a layer uses them, once
    eagerly and replayed from a graph captured on another stream: the same bits."""
    T, E, top, d, h = 300, 8, 2, 128, 256
    x0 = _rand((T, d), "bf16", 1)
    router = torch.randn((d, E), device="cuda", generator=_gen(2)) * d ** -0.5
    w1 = torch.randn((E, d, h), device="cuda", generator=_gen(3)).bfloat16() * d ** -0.5
    w2 = torch.randn((E, h, d), device="cuda", generator=_gen(4)).bfloat16() * h ** -0.5
    dout = _rand((T, d), "bf16", 5)
    x = x0.clone()

    def step():
        z = x.float() @ router
        r = G.route(z, top)
        rows = G.dispatch(x, r)
        hid = G.grouped_matmul(rows, w1, r.offsets, relu=True)
        y = G.grouped_matmul(hid, w2, r.offsets)
        out = G.combine(y, r, residual=x)
        dy, dw = G.combine_grad(dout, y, r)
        dh = G.grouped_matmul(dy, w2.transpose(1, 2), r.offsets) * (hid > 0)
        g1, g2 = G.grouped_weight_grad(rows, dh, r.offsets), G.grouped_weight_grad(hid, dy, r.offsets)
        drows = G.grouped_matmul(dh, w1.transpose(1, 2), r.offsets)
        dx = G.dispatch_grad(drows, r)
        dz = G.route_grad(z, r, dweights=dw, dloss=0.01)
        norm = G.clip_grad_norm([g1, g2], 0.5)
        return [out, dx, dz, g1, g2, norm, r.loss]

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.zero_()
    graph.replay()
    x.copy_(x0)
    graph.replay()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert G.default_plan_status() == 0


def test_refusals():
    r = _routing(10, 8, 2)
    x, y = _rand((10, 16), "f16", 1), _rand((20, 16), "f16", 2)
    for bad in (lambda: G.dispatch(x[:9], r), lambda: G.dispatch(x.double(), r), lambda: G.dispatch(x.t(), r),
                lambda: G.dispatch(x.cpu(), r), lambda: G.dispatch(x, r, out=y.float()),
                lambda: G.combine(y, r, residual=x[:9]), lambda: G.combine(y, r, residual=x.float()),
                lambda: G.combine(y, r._replace(weights=r.weights[:, :1])),
                lambda: G.combine(y, r._replace(slots=r.slots.long())), lambda: G.combine(y, r, out=y),
                lambda: G.combine_grad(x[:9], y, r), lambda: G.combine_grad(x.float(), y, r),
                lambda: G.combine_grad(x, y, r, out=y[:5])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(G.GemmError):
        G.combine_grad(x, y, r, out=y)
    with pytest.raises(G.GemmError):
        G.dispatch(x, r, plan=G.Plan(G.GEMM_BF16, G.GEMM_F32))
