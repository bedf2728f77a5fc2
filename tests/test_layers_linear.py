"""Fully connected layers (linear) and their gradients (linear_grad) against 64-bit forms, on
every path that they choose by size.

Bounds: a product of depth K is off by (K + 4) 2^-23 of the product of absolute values (fp32
sums that truncate), an activation by what layer_helpers derives, a result by half a step of
its type.  In the gradients dz is rounded to the operands' type: half a step of every term."""
import math

import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from layer_helpers import ACTS, DT, EPS, TINY, U, act_grad_error, act_ref, linear_ref, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _rand(shape, dtype, seed, scale=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=gen) * scale).to(DT[dtype])


def _layer(M, K, N, dtype, layout="kn", odd=False, seed=0):
    """x and w; odd: at pitches and addresses that TMA cannot take, NaN around them."""
    def place(v):
        if not odd:
            return v
        wide = torch.full((v.shape[0] + 1, v.shape[1] + 5), math.nan, device="cuda", dtype=v.dtype)
        wide[:-1, 3:3 + v.shape[1]] = v
        return wide[:-1, 3:3 + v.shape[1]]

    x = place(_rand((M, K), dtype, seed + 1))
    w = _rand((K, N), dtype, seed + 2, K ** -0.5 if K else 1.0)
    return x, place(w) if layout == "kn" else place(w.t().contiguous()).t()


def _check(x, w, act, bias, residual, out, dtype, save=True, **kw):
    r = G.linear(x, w, bias=bias, activation=act, residual=residual, save_pre=save, out_dtype=DT[out], **kw)
    y, pre = r if save else (r, None)
    ref, z, ey, ez = linear_ref(x, w, bias, act, residual)
    within(y, ref, U[out] * (ref.abs() + ey) + ey + TINY[out], "y")
    if save:
        within(pre, z, U[out] * (z.abs() + ez) + ez + TINY[out], "pre")


# (rows, K, N, rows of a tile and CTAs that share its K; 0: the tile kernel, on single CTAs or pairs)
SIZES = [(1, 64, 16, 16, 1), (1, 65, 128, 16, 1), (1, 4096, 11008, 16, 3), (7, 1024, 1000, 16, 4),
         (16, 200, 130, 16, 2), (17, 256, 384, 32, 2), (1, 128, 20000, 16, 1), (32, 8200, 1000, 32, 8),
         (33, 2048, 4096, 64, 4), (64, 512, 20000, 0, 0), (64, 4096, 20000, 64, 1), (60, 1030, 2000, 64, 4),
         (65, 320, 300, 64, 2), (65, 130, 300, 0, 0), (128, 1000, 2048, 64, 4), (129, 2050, 640, 64, 4),
         (300, 700, 1024, 64, 4), (128, 4100, 11000, 128, 3), (250, 9000, 7000, 128, 2), (1000, 1000, 2048, 0, 0),
         (200, 256, 12000, 0, 0), (513, 264, 9000, 0, 0)]


@pytest.mark.parametrize("M,K,N,box,splits", SIZES)
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype,act", [("bf16", "gelu"), ("f16", "silu")])
def test_linear(M, K, N, box, splits, layout, dtype, act):
    x, w = _layer(M, K, N, dtype, layout)
    bias, res = _rand((N,), "f32", 3, 0.3), _rand((M, N), dtype, 4)
    plan = G.Plan(G.DTYPE_CODES[dtype], G.GEMM_F32)
    _check(x, w, act, bias, res, dtype, dtype, plan=plan)
    c = plan.last_config()
    assert ((c["bn"], c["split_k"]) if c["bk"] == 64 else (0, 0)) == (box, splits) and plan.device_status() == 0


# Single CTAs and pairs of the tile kernel: rows of one and of several tiles, ragged last ones.
@pytest.mark.parametrize("M,K,N,cta_group", [(65, 130, 300, 1), (1000, 1000, 2048, 1), (520, 72, 12000, 1), (250, 4100, 19001, 2),
                                             (700, 2100, 6000, 2), (2040, 1990, 2100, 2), (3001, 640, 5000, 2)])
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32")])
def test_single_ctas_and_pairs(M, K, N, cta_group, layout, dtype, out):
    x, w = _layer(M, K, N, dtype, layout)
    plan = G.Plan(G.DTYPE_CODES[dtype], G.GEMM_F32)
    _check(x, w, "gelu", _rand((N,), "bf16", 3), _rand((M, N), out, 4), out, dtype, plan=plan)
    assert plan.last_config()["cta_group"] == cta_group and plan.device_status() == 0


@pytest.mark.parametrize("act", ACTS, ids=str)
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K,N", [(5, 96, 200), (260, 128, 10001)])
def test_activations_and_types(act, out, M, K, N):
    """Each activation over the range where it bends (z of deviation 3), each type of bias and result."""
    dtype = "f16" if out == "f16" else "bf16"
    x, w = _layer(M, K, N, dtype)
    x = x * 3
    _check(x, w, act, _rand((N,), out, 3), None, out, dtype)
    _check(x, w, act, None, _rand((M, N), out, 4), out, dtype, save=False)


@pytest.mark.parametrize("M,K,N", [(1, 63, 7), (3, 100, 129), (70, 77, 250), (200, 131, 4001), (300, 129, 20003)])
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_odd_sizes_pitches_and_addresses(M, K, N, layout, dtype):
    x, w = _layer(M, K, N, dtype, layout, odd=True)
    _check(x, w, "gelu_tanh", _rand((N,), dtype, 3), _rand((M, N), dtype, 4), dtype, dtype)
    wide = torch.full((M, N + 9), 7.0, device="cuda", dtype=DT[dtype])
    res = _rand((M, N + 3), dtype, 5)[:, 1:1 + N]
    out = G.linear(x, w, activation="silu", residual=res, out=wide[:, 3:3 + N])
    assert torch.equal(out, G.linear(x, w, activation="silu", residual=res))
    assert (wide[:, :3] == 7).all() and (wide[:, 3 + N:] == 7).all()


def test_the_residual_in_place_and_plain_calls():
    for M in (4, 400):
        x, w = _layer(M, 256, 9000, "bf16")
        res = _rand((M, 9000), "bf16", 4)
        want = G.linear(x, w, residual=res)
        assert G.linear(x, w, residual=res, out=res) is res and torch.equal(res, want)
        _check(x, w, None, None, None, "bf16", "bf16", save=False)


def test_empty_sizes():
    for M, K, N in ((0, 8, 8), (8, 8, 0), (3, 0, 40), (200, 0, 300)):
        x, w = torch.zeros((M, K), device="cuda", dtype=torch.float16), torch.zeros((K, N), device="cuda", dtype=torch.float16)
        b, res = _rand((N,), "f32", 1), _rand((M, N), "f16", 2)
        y, pre = G.linear(x, w, bias=b, activation="relu", residual=res, save_pre=True)
        within(y, b.double().clamp(min=0) + res.double(), 2.0 ** -11 * (b.abs() + res.abs()).double() + 1e-7)
        within(pre, b.double().expand(M, N), 2.0 ** -11 * b.abs().double().expand(M, N) + 1e-7)
        dx, dw, db = G.linear_grad(res, x, w, activation="silu", pre=pre)
        assert dx.shape == (M, K) and dw.shape == (K, N) and db.shape == (N,)
        assert (dx == 0).all() if N == 0 else True
        assert ((dw == 0).all() and (db == 0).all()) if M == 0 else True


def test_nan_and_infinity_go_their_way():
    """A row or a column that holds them spoils its own results only; ReLU keeps NaN."""
    for M in (6, 300):
        x, w = _layer(M, 128, 9000, "bf16")
        x[2, 5] = math.nan
        w[7, 77] = math.inf
        for act in ACTS:
            y = G.linear(x, w, activation=act)
            assert y[2].isnan().all()
            clean = torch.ones_like(y, dtype=torch.bool)
            clean[2], clean[:, 77] = False, False
            assert y[clean].isfinite().all()
            assert not y[[0, 1, 3], 77].isfinite().all()


@pytest.mark.parametrize("act", ACTS, ids=str)
def test_large_arguments(act):
    """z far out, up to what bf16 holds: no overflow in between."""
    x = torch.eye(64, device="cuda").bfloat16()
    for scale in (20.0, 100.0, 3e4, 1e25):
        w = _rand((64, 72), "bf16", 1, scale)
        _check(x, w, act, None, None, "f32", "bf16", save=False)
        z, dy = w, torch.ones_like(w)
        _, dw, db = G.linear_grad(dy, x, w, activation=act, pre=z, dw_dtype=torch.float32)
        _, d = act_ref(z.double().clamp(-100, 100), act)
        within(dw, d, 2.0 ** -8 * d.abs() + 2e-6 * 101, "derivative")
        assert db.isfinite().all()


@pytest.mark.parametrize("act", ACTS[1:])
def test_derivatives_at_infinity(act):
    """A z that has overflowed to infinity has the slope 1 or 0; NaN stays NaN."""
    pre = torch.zeros((3, 8), device="cuda").half()
    pre[:, 1], pre[:, 2], pre[1, 5] = math.inf, -math.inf, math.nan
    _, _, db = G.linear_grad(torch.ones_like(pre), torch.ones((3, 8), device="cuda").half(),
                             torch.ones((8, 8), device="cuda").half(), activation=act, pre=pre)
    at0 = 0.0 if act == "relu" else 0.5
    assert db[1] == 3 and db[2] == 0 and db[5].isnan() and abs(float(db[0]) - 3 * at0) < 1e-5


GRADS = [(1, 64, 16), (5, 200, 130), (64, 1024, 1000), (300, 512, 1368), (777, 130, 264), (129, 1000, 2999), (2000, 264, 200),
         (1030, 1100, 2050)]


@pytest.mark.parametrize("M,K,N", GRADS)
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype,act", [("bf16", "gelu"), ("f16", "gelu_tanh"), ("f16", None), ("bf16", "silu"), ("f16", "relu")])
@pytest.mark.parametrize("odd", [False, True])
def test_gradients(M, K, N, layout, dtype, act, odd):
    x, w = _layer(M, K, N, dtype, layout, odd)
    dy, pre = _rand((M, N), dtype, 3), _rand((M, N), dtype, 4, 1.5)
    if odd:
        wide = torch.full((M, N + 3), math.nan, device="cuda", dtype=DT[dtype])
        wide[:, 1:1 + N] = dy
        dy = wide[:, 1:1 + N]
        pre = torch.cat((pre, pre[:, :1]), 1)[:, :N]
    plan = G.Plan(G.DTYPE_CODES[dtype], G.GEMM_F32)
    dx, dw, db = G.linear_grad(dy, x, w, activation=act, pre=pre if act else None, plan=plan)
    assert dx.dtype is x.dtype and dw.dtype is w.dtype and dw.stride(1 if layout == "kn" else 0) == 1
    _, d = act_ref(pre.double(), act)
    dz = dy.double() * d
    step = (U[dtype] if act not in (None, "relu") else 0.0) * dz.abs() + dy.double().abs() * act_grad_error(pre.double(), act)
    tiny = TINY[dtype]
    for got, ref, mag, extra, depth in (
            (dx, dz @ w.double().t(), dz.abs() @ w.double().abs().t(), (step + tiny) @ w.double().abs().t(), N),
            (dw, x.double().t() @ dz, x.double().abs().t() @ dz.abs(), x.double().abs().t() @ (step + tiny), M)):
        e = (depth + 4) * EPS * mag + 1.01 * extra
        within(got, ref, U[dtype] * (ref.abs() + e) + e + tiny)
    e = (M + 4) * 2.0 ** -24 * dz.abs().sum(0) + (dy.double().abs() * act_grad_error(pre.double(), act)).sum(0)
    within(db, dz.sum(0), e + 1e-37, "db")
    assert plan.device_status() == 0
    # a part of them alone, and dw in fp32
    only = G.linear_grad(dy, x, w, activation=act, pre=pre if act else None, input_grad=False, bias_grad=False, dw_dtype=torch.float32)
    assert only[0] is None and only[2] is None
    within(only[1].to(DT[dtype]), dw, 1.01 * 2 * U[dtype] * dw.double().abs() + tiny)
    assert torch.equal(G.linear_grad(dy, x, w, activation=act, pre=pre if act else None, weight_grad=False)[0], dx)


@pytest.mark.parametrize("act", ACTS[1:])
def test_gradients_against_differences(act):
    """Differences of the 64-bit layer: loss = sum(c * y).  A step h of 1e-5 is off by 1e-10 times the
    third derivative and by 1e-16 / h of rounding; dz's rounding to fp16 is 2^-11 of each of its terms."""
    M, K, N, h = 3, 8, 8, 1e-5
    x, w = _layer(M, K, N, "f16", seed=5)
    b, c = _rand((N,), "f32", 3), _rand((M, N), "f16", 4)
    y, pre = G.linear(x, w, bias=b, activation=act, save_pre=True)
    pre64 = x.double() @ w.double() + b.double()
    if act == "relu":
        c = torch.where(pre64.abs() < 1e-2, 0.0, c.double()).half()   # (no difference across the kink)
    dx, dw, db = G.linear_grad(c, x, w, activation=act, pre=pre)

    def loss(x, w, b):
        return float((c.double() * act_ref(x @ w + b, act)[0]).sum())

    args = [x.double(), w.double(), b.double()]
    total = c.double().abs().sum()
    for i, got in enumerate((dx, dw, db)):
        for k in range(0, got.numel(), 5):
            up, down = [a.clone() for a in args], [a.clone() for a in args]
            up[i].view(-1)[k] += h
            down[i].view(-1)[k] -= h
            want = (loss(*up) - loss(*down)) / (2 * h)
            # dz and the result are rounded (2^-11 each), and pre is (2^-11, where the slope's own slope is below 2)
            assert abs(want - float(got.reshape(-1)[k])) < 6 * 2.0 ** -11 * (abs(want) + float(total) * 0.5), (act, i, k)


@pytest.mark.parametrize("M", [3, 250])
def test_layers_together_in_a_graph_and_on_another_stream(M):
    """Two layers with a residual, forward and backward, eagerly and replayed from a graph captured
    on another stream; two calls in it share the plan's scratch.  The same bits, and every replay
    follows its input."""
    d, h = 190, 517   # (operands that TMA cannot address: scratch everywhere)
    x0 = _rand((M, d), "bf16", 1)
    w1, w2 = _rand((d, h), "bf16", 2, d ** -0.5), _rand((h, d), "bf16", 3, h ** -0.5)
    b1, dy = _rand((h,), "f32", 4), _rand((M, d), "bf16", 5)
    x = x0.clone()
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)

    def step():
        hid, z = G.linear(x, w1, bias=b1, activation="gelu", save_pre=True, plan=plan)
        y = G.linear(hid, w2, residual=x, plan=plan)
        dh, dw2, _ = G.linear_grad(dy, hid, w2, bias_grad=False, plan=plan)
        dx, dw1, db1 = G.linear_grad(dh, x, w1, activation="gelu", pre=z, plan=plan)
        return [y, dw2, dx, dw1, db1, G.clip_grad_norm([dw1, dw2, db1], 1.0, plan=plan)]

    want = [t.clone() for t in step()]
    x.mul_(2)
    other = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for scale, ref in ((1, want), (2, other), (1, want)):
        x.copy_(x0 * scale)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert plan.device_status() == 0


def test_a_layer_past_four_gigabytes():
    """Offsets past 32 bits in every operand that is as large as the result: 70000 x 40000 entries of
    bf16; the first, middle and last rows."""
    M, K, N = 70000, 64, 40000
    x, w = _layer(M, K, N, "bf16")
    res = torch.randn((M, N), device="cuda", generator=torch.Generator("cuda").manual_seed(5)).bfloat16()
    y, pre = G.linear(x, w, activation="gelu", residual=res, save_pre=True)
    rows = [0, 1, M // 2, M - 2, M - 1]
    ref, z, ey, ez = linear_ref(x[rows], w, None, "gelu", res[rows])
    within(y[rows], ref, U["bf16"] * (ref.abs() + ey) + ey, "y")
    within(pre[rows], z, U["bf16"] * (z.abs() + ez) + ez, "pre")
    del y
    dx, _, db = G.linear_grad(res, x, w, activation="gelu", pre=pre, weight_grad=False)
    _, d = act_ref(pre[rows].double(), "gelu")
    dz = res[rows].double() * d
    step = U["bf16"] * dz.abs() + res[rows].double().abs() * act_grad_error(pre[rows].double(), "gelu")
    ref, wd = dz @ w.double().t(), w.double().abs().t()
    e = (N + 4) * EPS * (dz.abs() @ wd) + 1.01 * (step @ wd)
    within(dx[rows], ref, U["bf16"] * (ref.abs() + e) + e, "dx")
    cols = [0, 20000, N - 1]
    _, d = act_ref(pre[:, cols].double(), "gelu")
    dz = res[:, cols].double() * d
    e = (M + 4) * 2.0 ** -24 * dz.abs().sum(0) + (res[:, cols].double().abs() * act_grad_error(pre[:, cols].double(), "gelu")).sum(0)
    within(db[cols], dz.sum(0), e, "db")


def test_a_forced_kernel_is_for_other_calls():
    """set_kernel is gemm_run's: the layers choose for themselves and leave it as it was."""
    x, w = _layer(100, 264, 200, "f16")
    dy = _rand((100, 200), "f16", 3)
    plan = G.Plan(G.GEMM_F16, G.GEMM_F32)
    want = G.linear_grad(dy, x, w, plan=plan)
    plan.set_kernel(G.GEMM_KERNEL_SIMT)
    got = G.linear_grad(dy, x, w, plan=plan)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    G.matmul(x, w, plan=plan)
    assert plan.last_config()["kernel"] == G.GEMM_KERNEL_SIMT


@pytest.mark.parametrize("planned", [False, True])
def test_calls_on_two_streams_at_once(planned):
    """Two layers on two streams behind queued work, with default plans or one each: their scratch
    (operands that TMA cannot address, dz) is not shared."""
    sets = []
    for i in range(2):
        x, w = _layer(300 + 40 * i, 131, 517, "bf16", seed=10 * i)
        sets.append((x, w, _rand((x.shape[0], 517), "bf16", 5 + i), _rand((x.shape[0], 517), "bf16", 7 + i)))
    plans = [G.Plan(G.GEMM_BF16, G.GEMM_F32) if planned else None for _ in range(2)]

    def run(i):
        x, w, dy, pre = sets[i]
        y = G.linear(x, w, activation="gelu", residual=dy, plan=plans[i])
        return [y, *G.linear_grad(dy, x, w, activation="gelu", pre=pre, plan=plans[i])]

    want = [[t.clone() for t in run(i)] for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            torch.cuda._sleep(50_000_000)
    for turn in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, run(i)))
    torch.cuda.synchronize()
    for i, r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


@pytest.mark.parametrize("M,N", [(5, 4096), (600, 9000)])
def test_expired_waits_are_reported_and_the_plan_survives(M, N):
    x, w = _layer(M, 8192, N, "f16")
    plan = G.Plan(G.GEMM_F16, G.GEMM_F32)
    want = G.linear(x, w, activation="gelu", plan=plan)
    G.gemm_plan_set_timeout(plan.handle, 200)       # 200 ns
    for _ in range(3):
        G.linear(x, w, activation="gelu", plan=plan)
    # (a wait whose first try is granted does not expire: the hardware suspends it for a while)
    assert plan.device_status() in (0, G.GEMM_ERR_TIMEOUT)
    G.gemm_plan_set_timeout(plan.handle, 4_000_000_000)
    assert torch.equal(G.linear(x, w, activation="gelu", plan=plan), want) and plan.device_status() == 0


def test_refusals():
    x, w = _layer(4, 64, 32, "f16")
    dy = _rand((4, 32), "f16", 1)
    for bad in (lambda: G.linear(x, w[:60]), lambda: G.linear(x, w.float()), lambda: G.linear(x.float(), w.float(), activation="tanh"),
                lambda: G.linear(x, w, activation="tanh"), lambda: G.linear(x.t(), w.t()), lambda: G.linear(x, w[:, ::2]),
                lambda: G.linear(x.cpu(), w.cpu()), lambda: G.linear(x, w, bias=torch.zeros(31, device="cuda")),
                lambda: G.linear(x, w, bias=torch.zeros(32, device="cuda", dtype=torch.float64)),
                lambda: G.linear(x, w, residual=dy.float()), lambda: G.linear(x, w, residual=dy[:3]),
                lambda: G.linear(x, w, out=torch.zeros((4, 33), device="cuda", dtype=torch.float16)),
                lambda: G.linear(x, w, out_dtype=torch.int32), lambda: G.linear_grad(dy, x, w, activation="gelu"),
                lambda: G.linear_grad(dy.float(), x, w), lambda: G.linear_grad(dy[:3], x, w),
                lambda: G.linear_grad(dy, x, w, activation="gelu", pre=dy.float()),
                lambda: G.linear_grad(dy, x, w, dw_dtype=torch.int8)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(G.GemmError):
        G.linear(x.float(), w.float())
    with pytest.raises(G.GemmError):
        G.linear(x, w, plan=G.Plan(G.GEMM_BF16, G.GEMM_F32))
