"""Routing of tokens to experts, its balance loss and its gradient, against 64-bit forms.

Choices, places and counts are compared for equality.  Bounds of the rest: a probability is
a quotient of exponentials, (8 + 2 spread) 2^-23 of its value with the rounding of the
arguments (spread: the widest row of logits) and of the warp's sum; sums over the tokens of a
warp add as many 2^-24."""
import math

import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from layer_helpers import DT, EPS, U, route_grad_ref, route_ref, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _logits(tokens, experts, dtype, seed, scale=1.5):
    gen = torch.Generator("cuda").manual_seed(seed)
    return (scale * torch.randn((tokens, experts), device="cuda", generator=gen)).to(DT[dtype])


def _check(z, top, renormalize=True, mask=None, r=None, **kw):
    r = r or G.route(z, top, renormalize=renormalize, mask=mask, **kw)
    w, experts, slots, counts, offsets, routed, loss, p, spread = route_ref(z, top, renormalize, mask)
    for got, want in ((r.experts, experts), (r.slots, slots), (r.counts, counts), (r.offsets, offsets)):
        assert got.dtype is torch.int32 and torch.equal(got.long().cpu(), want)
    assert int(r.routed) == routed
    rel = (8 + 2 * spread) * EPS
    within(r.weights.cpu(), w, 2 * rel * w.abs() + 1e-37, "weights")
    within(r.loss.cpu(), loss, (rel + (z.shape[0] + 16) * 2.0 ** -24) * loss.abs() + 1e-37, "loss")
    return r


SIZES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (16, 8, 2), (64, 64, 6), (65, 33, 4), (257, 32, 8), (1000, 64, 1),
         (300, 100, 7), (90, 160, 6), (77, 257, 32), (130, 512, 8), (70, 1000, 9), (66, 1024, 32), (4097, 16, 3), (150000, 12, 2), (700, 1023, 3)]


@pytest.mark.parametrize("tokens,experts,top", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_route(tokens, experts, top, dtype):
    z = _logits(tokens, experts, dtype, tokens)
    _check(z, top, renormalize=dtype != "f16")


@pytest.mark.parametrize("tokens,experts,top", [(40, 8, 2), (700, 40, 4), (2500, 64, 6)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_padded_tokens_and_closed_experts(tokens, experts, top, renormalize):
    """Masked tokens; experts at -inf for all, for some, and for every but one; a row of nothing
    but -inf; rows of the type's lowest value."""
    z = _logits(tokens, experts, "f32", 2)
    z[:, 3] = -math.inf
    z[1::7, ::2] = -math.inf
    z[2] = -math.inf
    z[4, :] = -math.inf
    z[4, 5] = 1.0
    z[6] = torch.finfo(torch.float32).min
    z[7, 1:] = torch.finfo(torch.float32).min
    z[8, :] = -0.0
    z[8, 1::2] = 0.0
    mask = torch.ones(tokens, dtype=torch.bool, device="cuda")
    mask[5::11] = False
    r = G.route(z, top, renormalize=renormalize, mask=mask)
    # (rows that hold the lowest value: their other probabilities are 0, the spread of the rest counts)
    w, experts_, slots, counts, offsets, routed, loss, p, _ = route_ref(z, top, renormalize, mask)
    assert torch.equal(r.experts.long().cpu(), experts_) and torch.equal(r.slots.long().cpu(), slots)
    assert torch.equal(r.counts.long().cpu(), counts) and torch.equal(r.offsets.long().cpu(), offsets)
    assert int(r.routed) == routed
    rel = (8 + 2 * 16) * EPS
    within(r.weights.cpu(), w, 2 * rel * w.abs() + 1e-37, "weights")
    within(r.loss.cpu(), loss, (rel + (tokens + 16) * 2.0 ** -24) * loss.abs(), "loss")


@pytest.mark.parametrize("tokens", [1, 50, 3000])
def test_nothing_is_routed(tokens):
    z = _logits(tokens, 8, "f32", 1)
    r = _check(z, 2, mask=torch.zeros(tokens, dtype=torch.uint8, device="cuda"))
    assert float(r.loss) == 0 and int(r.routed) == 0
    d = G.route_grad(z, r, dweights=torch.ones((tokens, 2), device="cuda"), dloss=3.0)
    assert (d == 0).all()
    r = _check(torch.full_like(z, -math.inf), 2)
    assert (r.slots == -1).all()


def test_no_tokens():
    r = G.route(torch.empty((0, 8), device="cuda"), 2)
    assert r.weights.shape == (0, 2) and (r.counts == 0).all() and (r.offsets == 0).all()
    assert float(r.loss) == 0 and int(r.routed) == 0
    assert G.route_grad(torch.empty((0, 8), device="cuda"), r, dloss=1.0).shape == (0, 8)
    assert G.dispatch(torch.empty((0, 16), device="cuda"), r).shape == (0, 16)
    assert G.combine(torch.empty((0, 16), device="cuda"), r).shape == (0, 16)
    dy, dw = G.combine_grad(torch.empty((0, 16), device="cuda"), torch.empty((0, 16), device="cuda"), r)
    assert dy.shape == (0, 16) and dw.shape == (0, 2)


@pytest.mark.parametrize("tokens", [30, 900])
def test_ties_go_to_the_lower_index(tokens):
    z = torch.randint(-1, 2, (tokens, 48), device="cuda", generator=torch.Generator("cuda").manual_seed(4)).bfloat16()
    _check(z, 7)
    _check(torch.zeros_like(z), 3)


def test_nan_and_infinity_stay_visible():
    z = _logits(200, 16, "f32", 5)
    z[3, 9] = math.nan
    z[5, 2] = z[5, 11] = -math.nan
    z[7, 1] = math.inf
    r = G.route(z, 4)
    w, experts, slots, counts, *_ = route_ref(z, 4)
    assert torch.equal(r.experts.long().cpu(), experts) and torch.equal(r.slots.long().cpu(), slots)
    assert torch.equal(r.counts.long().cpu(), counts)
    assert r.weights[[3, 5, 7]].isnan().all() and r.loss.isnan()
    rest = torch.ones(200, dtype=torch.bool)
    rest[[3, 5, 7]] = False
    within(r.weights.cpu()[rest], w[rest], 1e-5 * w[rest])
    d = G.route_grad(z, r, dweights=torch.ones((200, 4), device="cuda"), dloss=1.0).cpu()
    assert d[[3, 5, 7]].isnan().all() and not d[rest].isnan().any()


@pytest.mark.parametrize("tokens,experts,top", [(20, 8, 2), (500, 37, 5)])
def test_strides_and_kept_buffers(tokens, experts, top):
    """Logits inside wider rows (whose other entries are NaN), and a routing written again."""
    wide = torch.full((tokens, experts + 11), math.nan, device="cuda")
    wide[:, 3:3 + experts] = _logits(tokens, experts, "f32", 6)
    z = wide[:, 3:3 + experts]
    r = _check(z, top)
    other = _logits(tokens, experts, "f32", 7)
    kept = G.route(other, top, out=r)
    assert kept.weights is r.weights
    _check(other, top, r=r)
    d = torch.full((tokens, experts + 5), 7.0, device="cuda")
    G.route_grad(other, r, dloss=2.0, out=d[:, 2:2 + experts])
    assert torch.equal(d[:, 2:2 + experts], G.route_grad(other, r, dloss=2.0))
    assert (d[:, :2] == 7).all() and (d[:, 2 + experts:] == 7).all()


@pytest.mark.parametrize("tokens,experts,top", [(9, 5, 3), (64, 8, 2), (65, 33, 4), (2000, 100, 6), (300, 1024, 5)])
def test_nothing_is_written_around_a_routing(tokens, experts, top):
    z = _logits(tokens, experts, "f32", 3)
    f = torch.full((tokens * top + 9,), 7.0, device="cuda")
    i = torch.full((2 * tokens * top + 2 * experts + 40,), 7, dtype=torch.int32, device="cuda")
    at, views = 4, []
    for n, shape in ((tokens * top, (tokens, top)), (tokens * top, (tokens, top)), (experts, (experts,)),
                     (experts + 1, (experts + 1,)), (1, ())):
        views.append(i[at:at + n].view(shape))
        at += n + 4
    out = G.Routing(f[4:4 + tokens * top].view(tokens, top), *views, f[-1:].view(()))
    guard = torch.ones_like(i, dtype=torch.bool)
    at = 4
    for n in (tokens * top, tokens * top, experts, experts + 1, 1):
        guard[at:at + n] = False
        at += n + 4
    _check(z, top, r=G.route(z, top, out=out))
    assert (i[guard] == 7).all() and (f[:4] == 7).all() and (f[4 + tokens * top:-1] == 7).all()


@pytest.mark.parametrize("tokens,experts,top", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient(tokens, experts, top, dtype, renormalize):
    z = _logits(tokens, experts, dtype, tokens + 1)
    z[::5, experts // 2] = -math.inf if experts > 1 else z[::5, 0]
    mask = torch.arange(tokens, device="cuda") % 9 != 4
    gen = torch.Generator("cuda").manual_seed(3)
    dw = torch.randn((tokens, top), device="cuda", generator=gen)
    r = G.route(z, top, renormalize=renormalize, mask=mask)
    dw = torch.where(r.experts < 0, math.nan, dw)   # what belongs to no expert is not read
    dloss = torch.full((1,), 0.3 * tokens, device="cuda")
    for use_w, use_l in ((True, True), (False, True), (True, False)):
        got = G.route_grad(z, r, dweights=dw if use_w else None, dloss=dloss if use_l else None)
        assert got.dtype is z.dtype
        ref, mag, spread = route_grad_ref(z, top, dw.nan_to_num(0.0) if use_w else None, 0.3 * tokens if use_l else 0.0,
                                          renormalize, mask)
        rel = (24 + experts / 32 + 4 * spread) * EPS
        within(got.cpu(), ref, U[dtype] * ref.abs() + rel * (1 + U[dtype]) * mag + (2.0 ** -24 if dtype == "f16" else 1e-37))
    twice = G.route_grad(z, r, dloss=0.3 * tokens)
    assert torch.equal(twice, G.route_grad(z, r, dloss=dloss))


@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_against_differences(renormalize):
    """Central differences of the 64-bit loss and weights: a step h is off by h^2 / 6 of the third
    derivative (below 10 here), 2e-8 for h = 1e-4, and 1e-12 / h of rounding; fp32 adds 1e-6."""
    T, E, top, h = 6, 5, 2, 1e-4
    z = _logits(T, E, "f32", 12)
    dw = torch.randn((T, top), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    d = G.route_grad(z, G.route(z, top, renormalize=renormalize), dweights=dw, dloss=2.5).double().cpu()

    def value(x):
        w, _, _, _, _, _, loss, _, _ = route_ref(x, top, renormalize)
        return float((w * dw.double().cpu()).sum() + 2.5 * loss)

    zd = z.double().cpu()
    for t in range(T):
        for e in range(E):
            up, down = zd.clone(), zd.clone()
            up[t, e] += h
            down[t, e] -= h
            assert abs((value(up) - value(down)) / (2 * h) - float(d[t, e])) < 1e-5


def test_logits_past_four_gigabytes():
    """2.2 million tokens by 1000 experts in fp16: offsets past 32 bits; the last tokens' choices,
    weights and gradients, and the counts of all."""
    T, E, top, n = 2_200_000, 1000, 2, 50
    z = torch.empty((T, E), device="cuda", dtype=torch.float16)
    for i in range(0, T, 200_000):
        z[i:i + 200_000] = torch.randn((200_000, E), device="cuda", generator=torch.Generator("cuda").manual_seed(i)).half()
    r = G.route(z, top)
    w, experts, *_, spread = route_ref(z[-n:], top)
    assert torch.equal(r.experts[-n:].long().cpu(), experts)
    within(r.weights[-n:].cpu(), w, 2 * (8 + 2 * spread) * EPS * w, "weights")
    assert torch.equal(r.counts.long(), torch.bincount(r.experts.flatten().long(), minlength=E))
    assert int(r.offsets[-1]) == T * top and int(r.routed) == T
    place = torch.argsort(r.experts.flatten().long(), stable=True)
    assert torch.equal(r.slots.flatten()[place].long(), torch.arange(T * top, device="cuda"))
    dw = torch.randn((T, top), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    d = G.route_grad(z, r, dweights=dw)[-n:].double().cpu()
    ref, mag, spread = route_grad_ref(z[-n:], top, dw[-n:], 0.0)
    within(d, ref, U["f16"] * ref.abs() + (24 + E / 32 + 4 * spread) * EPS * (1 + U["f16"]) * mag + 2.0 ** -24)


def test_gradient_over_the_logits():
    z = _logits(333, 24, "bf16", 8)
    r = G.route(z, 3)
    want = G.route_grad(z, r, dloss=5.0)
    assert G.route_grad(z, r, dloss=5.0, out=z) is z and torch.equal(z, want)


def test_equal_bits_and_an_even_routing():
    z = _logits(5000, 64, "f32", 9)
    a, b = G.route(z, 6), G.route(z, 6)
    assert all(torch.equal(u, v) for u, v in zip(a[:7], b[:7]))
    even = torch.eye(16, device="cuda").repeat(10, 1) * 50   # each expert as often as the others
    assert abs(float(G.route(even, 1).loss) - 1) < 1e-5


@pytest.mark.parametrize("tokens", [30, 2000])
def test_in_a_graph_and_on_another_stream(tokens):
    """A replay follows its inputs; two routings in one graph share the plan's scratch."""
    z, z2 = _logits(tokens, 32, "f32", 1), _logits(tokens, 32, "f32", 2)
    a, b = z.clone(), z2.clone()
    plan = G.Plan(G.GEMM_F32, G.GEMM_F32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r1, r2 = G.route(a, 4, plan=plan), G.route(b, 2, plan=plan)
        G.route_grad(a, r1, dloss=1.0, plan=plan)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r1, r2 = G.route(a, 4, plan=plan), G.route(b, 2, plan=plan)
        d = G.route_grad(a, r1, dloss=1.0, plan=plan)
    for swap in (False, True):
        a.copy_(z2 if swap else z)
        b.copy_(z if swap else z2)
        graph.replay()
        _check(a, 4, r=r1)
        _check(b, 2, r=r2)
        assert torch.equal(d, G.route_grad(a, r1, dloss=1.0))
    assert plan.device_status() == 0


def test_refusals():
    z = _logits(10, 8, "f32", 1)
    r = G.route(z, 2)
    for bad in (lambda: G.route(z, 0), lambda: G.route(z, 9), lambda: G.route(z.t(), 2), lambda: G.route(z.double(), 2),
                lambda: G.route(z.cpu(), 2), lambda: G.route(z, 2, mask=torch.ones(9, dtype=torch.bool, device="cuda")),
                lambda: G.route(z, 2, mask=torch.ones(10, device="cuda")), lambda: G.route(z, 3, out=r),
                lambda: G.route(z[:9], 2, out=r), lambda: G.route_grad(z[:9], r), lambda: G.route_grad(z[:, :7], r),
                lambda: G.route_grad(z, r, dweights=torch.ones((10, 3), device="cuda")),
                lambda: G.route_grad(z, r, dweights=torch.ones((10, 2), device="cuda").half()),
                lambda: G.route_grad(z, r, dloss=torch.ones(2, device="cuda")),
                lambda: G.route_grad(z, r, out=z.half())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: G.route(torch.zeros((4, 1025), device="cuda"), 2), lambda: G.route(torch.zeros((4, 64), device="cuda"), 33),
                lambda: G.route(z, 2, plan=G.Plan(G.GEMM_BF16, G.GEMM_F32))):
        with pytest.raises(G.GemmError):
            bad()
