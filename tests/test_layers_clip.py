"""The global norm of many tensors and clipping, against 64-bit forms.

The norm: squares are added in fp32 over 32 entries, which loses at most 33 2^-24 of a sum,
half of that of its root, then in fp64; it is rounded to fp32: 20 2^-24 of its value at most.  A scaled entry:
the factor is rounded once, the product twice: 2 2^-24 and half a step of the type."""
import math

import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from layer_helpers import DT, TINY, U, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _rand(shape, dtype, seed, scale=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=gen) * scale).to(DT[dtype])


def _norm(tensors):
    return math.sqrt(sum(float(t.double().square().sum()) for t in tensors))


def _check_norm(got, ref):
    assert got.shape == () and got.dtype is torch.float32
    if ref >= 2.0 ** 128:   # fp32 holds no such number
        assert float(got) == math.inf
        return
    # (2^-150: half of fp32's smallest step, what rounding a norm below 2^-126 may cost)
    assert abs(float(got) - ref) <= 20 * 2.0 ** -24 * ref + 2.0 ** -150, (float(got), ref)


def _check(tensors, max_norm, eps=1e-6, out=None):
    before = [t.clone() for t in tensors]
    ref = _norm(before)
    scale = min(1.0, max_norm / (ref + eps))
    norm = G.clip_grad_norm(tensors if out is None else G.TensorList(tensors, out=out), max_norm, eps=eps)
    _check_norm(norm, ref)
    for a, b in zip(out or tensors, before):
        want = b.double() * scale
        name = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}[a.dtype]
        within(a, want, (U[name] + 24 * 2.0 ** -24) * want.abs() + TINY[name], "scaled")
    if out is not None:
        assert all(torch.equal(a, b) for a, b in zip(tensors, before))


@pytest.mark.parametrize("shapes", [[(1,)], [(7,), (0,), (3, 5)], [(1000, 77)], [(8, 33, 129)] * 3 + [(5,)] * 40,
                                    [(4096,)], [(4097,)], [(2, 3, 1000, 501)], [(i % 67 + 1,) for i in range(1500)]],
                         ids=lambda s: f"{len(s)}-{s[0]}")
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_clip_in_place(shapes, dtype):
    t = [_rand(s, dtype, i) for i, s in enumerate(shapes)]
    n = _norm(t)
    _check(t, 0.3 * n)
    _check(t, 5 * n)
    _check(t, math.inf)


@pytest.mark.parametrize("src,dst", [("f32", "bf16"), ("f32", "f16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("start", [0, 1, 3])
def test_clip_into_other_buffers(src, dst, start):
    """Tensors at any element of a buffer, scaled into others at other alignments: the entries around
    them stay."""
    sizes = [1, 8, 31, 4096, 10000, 70001]
    bs, bd, t, o = [], [], [], []
    for i, n in enumerate(sizes):
        bs.append(_rand((n + 8,), src, i))
        bd.append(torch.full((n + 9,), 3.0, device="cuda", dtype=DT[dst]))
        t.append(bs[-1][start:start + n])
        o.append(bd[-1][2 * start:2 * start + n])
    for factor in (0.1, 3.0):
        _check(t, factor * _norm(t), out=o)
    for b, n in zip(bd, sizes):
        assert (b[:2 * start] == 3).all() and (b[2 * start + n:] == 3).all()


def test_mixed_types_and_orders():
    t = [_rand((64, 33), "f32", 1), _rand((40, 50), "bf16", 2).t(), _rand((6, 7, 8), "f16", 3).permute(2, 0, 1), _rand((), "f32", 4)]
    _check(t, 1.0)
    out = [torch.empty_like(x) for x in t]
    _check(t, 0.2, out=out)


@pytest.mark.parametrize("value", [1e-30, 3e-23, 1e-42, 1e25, 3e36])
@pytest.mark.parametrize("n", [1, 3, 20000])
def test_entries_of_any_size(value, n):
    """Squares that fp32 does not hold count all the same."""
    t = [torch.full((n,), value, device="cuda"), torch.zeros(100, device="cuda")]
    ref = _norm(t)
    _check_norm(G.grad_norm(t), ref)
    mixed = [torch.full((n,), value, device="cuda"), torch.full((5,), 2.0, device="cuda")]
    _check_norm(G.grad_norm(mixed), _norm(mixed))
    mixed = [torch.tensor([1e-25, 1.0, 1e30, 0.0, 1e-40, 5.0, 7.0, 2e20], device="cuda")]
    _check_norm(G.grad_norm(mixed), _norm(mixed))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_norm_that_is_not_finite_changes_nothing(bad, dtype):
    t = [_rand((5000,), dtype, 1), _rand((300,), dtype, 2)]
    t[1][77] = bad
    before = [x.clone() for x in t]
    norm = float(G.clip_grad_norm(t, 0.1))
    assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
    for a, b in zip(t, before):
        within(a, b, 0.0)
    out = [torch.empty_like(x) for x in t]
    G.clip_grad_norm(G.TensorList(t, out=out), 0.1)
    for a, b in zip(out, before):
        within(a, b, 0.0)


def test_zeros_empty_lists_and_a_bound_of_zero():
    z = [torch.zeros(1000, device="cuda"), torch.zeros((0, 4), device="cuda")]
    assert float(G.clip_grad_norm(z, 1.0)) == 0 and float(G.clip_grad_norm(z, 0.0, eps=0.0)) == 0
    assert (z[0] == 0).all()
    assert float(G.clip_grad_norm([], 1.0)) == 0 and float(G.grad_norm([])) == 0
    t = [_rand((999,), "f32", 1)]
    assert float(G.clip_grad_norm(t, 0.0)) > 0 and (t[0] == 0).all()


def test_norm_only_leaves_the_tensors():
    t = [_rand((12345,), "bf16", 1), _rand((77,), "f32", 2)]
    before = [x.clone() for x in t]
    _check_norm(G.grad_norm(t), _norm(t))
    _check_norm(G.grad_norm(G.TensorList(t, out=[torch.zeros_like(x) for x in t])), _norm(t))
    assert all(torch.equal(a, b) for a, b in zip(t, before))


def test_a_tensor_past_four_gigabytes():
    t = torch.zeros(2 ** 31 + 100, device="cuda", dtype=torch.bfloat16)
    t[-50:] = 2.0
    t[5] = 1.0
    _check_norm(G.clip_grad_norm([t], 1.0, eps=0.0), math.sqrt(201))
    assert abs(float(t[-1]) * math.sqrt(201) - 2) < 2 * 2.0 ** -8 and float(t[2 ** 30]) == 0
    del t


def test_equal_bits_graphs_and_streams():
    base = [_rand((300, 1000), "f32", 1), _rand((77777,), "bf16", 2)]
    runs = []
    for _ in range(2):
        t = [x.clone() for x in base]
        runs.append([G.clip_grad_norm(t, 1.0)] + t)
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    t = [x.clone() for x in base]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        G.clip_grad_norm([x.clone() for x in base], 1.0)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = G.clip_grad_norm(t, 1.0)   # (its list of addresses is the graph's own)
    for _ in range(2):
        for a, b in zip(t, base):
            a.copy_(b)
        graph.replay()
        assert torch.equal(norm, runs[0][0]) and all(torch.equal(a, b) for a, b in zip(t, runs[0][1:]))


def test_refusals():
    a = torch.zeros(100, device="cuda")
    for bad in (lambda: G.clip_grad_norm([a], -1.0), lambda: G.clip_grad_norm([a], math.nan), lambda: G.clip_grad_norm([a], 1.0, eps=-1.0),
                lambda: G.clip_grad_norm([a], 1.0, eps=math.inf), lambda: G.clip_grad_norm([a.double()], 1.0),
                lambda: G.clip_grad_norm([a.cpu()], 1.0), lambda: G.clip_grad_norm([a, a], 1.0),
                lambda: G.clip_grad_norm([a[:60], a[50:]], 1.0), lambda: G.clip_grad_norm([a[::2]], 1.0),
                lambda: G.clip_grad_norm([a[:1].expand(5)], 1.0), lambda: G.TensorList([a], out=[]),
                lambda: G.TensorList([a], out=[torch.zeros(99, device="cuda")]), lambda: G.TensorList([a[:50]], out=[a[10:60]])):
        with pytest.raises(ValueError):
            bad()
    moved = torch.zeros(100, device="cuda")
    kept = G.TensorList([moved])
    G.clip_grad_norm(kept, 1.0)
    moved.data = torch.zeros(100, device="cuda")
    with pytest.raises(ValueError):
        G.clip_grad_norm(kept, 1.0)
    G.TensorList([a[:50], a[:50]], out=[torch.zeros(50, device="cuda"), torch.zeros(50, device="cuda")])
