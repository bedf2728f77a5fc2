"""Products grouped by expert (gemm_run_grouped, gemm_run_grouped_wgrad) against
plain 64-bit forms: ragged and empty groups, rows of no group, odd widths,
strided and misaligned operands, both layouts of the weights, every type, the
fused epilogue, accumulation, and that a gradient is what differences give."""
import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from expert_helpers import DT, check, grouped_ref, offsets_of, wgrad_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


# rows of each group; K; N
SHAPES = [
    ([1], 64, 64),
    ([1, 0, 0, 2], 8, 8),
    ([0, 0, 0], 128, 128),
    ([5, 0, 17, 3], 200, 72),
    ([130, 1, 0, 256, 127], 320, 384),
    ([300], 1000, 520),
    ([255, 257, 513, 16, 15, 33], 136, 1000),
    ([64] * 40, 64, 256),
    ([3, 600], 1, 1),
    ([40, 0, 25], 33, 65),
    ([129, 64], 255, 257),
    ([2, 1], 4096, 16),
    ([700, 90], 2048, 264),
]


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("counts,K,N", SHAPES, ids=lambda v: str(v)[:24])
def test_grouped_matmul(counts, K, N, dtype, layout):
    gen = _gen(1)
    R, E = sum(counts), len(counts)
    x = _randn(gen, R, K, dtype=DT[dtype])
    w = _randn(gen, E, K, N, dtype=DT[dtype]) if layout == "kn" else _randn(gen, E, N, K, dtype=DT[dtype]).transpose(1, 2)
    off = offsets_of(counts)
    plan = G.Plan(G.DTYPE_CODES[dtype], G.GEMM_F32)
    for out in ("f32", dtype):
        y = G.grouped_matmul(x, w, off, out_dtype=DT[out], plan=plan)
        assert plan.device_status() == 0
        ref, mag = grouped_ref(x, w, off)
        check(y, ref, mag, K, out)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("relu", [False, True])
@pytest.mark.parametrize("bias", [None, "group", "shared"])
@pytest.mark.parametrize("N", [64, 203, 520])
def test_grouped_epilogue(N, bias, relu, out):
    gen = _gen(2)
    counts, K = [70, 0, 9, 300], 96
    x, w = _randn(gen, sum(counts), K, dtype=DT["bf16"]), _randn(gen, 4, K, N, dtype=DT["bf16"])
    b = None if bias is None else _randn(gen, 4, N) if bias == "group" else _randn(gen, N, dtype=DT["f16"])
    off = offsets_of(counts)
    y = G.grouped_matmul(x, w, off, alpha=-0.75, bias=b, relu=relu, out_dtype=DT[out])
    check(y, *grouped_ref(x, w, off, b, relu, -0.75), K, out)


@pytest.mark.parametrize("K,N", [(128, 256), (120, 88), (57, 61)])
def test_rows_of_no_group_and_foreign_nans(K, N):
    """Rows outside every group are not written, and NaN or infinity in one
    group's rows and weights or in rows of no group never reach another group."""
    gen = _gen(3)
    R, counts, first = 400, [100, 0, 77, 60], 33
    off = offsets_of(counts, first)
    o = off.tolist()
    x, w = _randn(gen, R, K, dtype=DT["f16"]), _randn(gen, 4, K, N, dtype=DT["f16"])
    dy = _randn(gen, R, N, dtype=DT["f16"])
    for t in (x, dy):
        t[:o[0]] = float("nan")
        t[o[4]:] = float("inf")
        t[o[2]:o[3]] = float("nan")    # group 2
    w[1] = float("nan")                # the empty group's weights
    out = torch.full((R, N), 7.0, device="cuda", dtype=DT["f32"])
    G.grouped_matmul(x, w, off, out=out)
    assert (out[:o[0]] == 7).all() and (out[o[4]:] == 7).all()
    assert out[o[2]:o[3]].isnan().all()
    ref, mag = grouped_ref(x, w, off)
    for g in (0, 3):
        s = slice(o[g], o[g + 1])
        check(out[s], ref[s], mag[s], K, "f32")
    dw = G.grouped_weight_grad(x, dy, off, out_dtype=DT["f32"])
    ref, mag = wgrad_ref(x, dy, off)
    assert dw[2].isnan().all() and (dw[1] == 0).all()
    for g in (0, 3):
        check(dw[g], ref[g], mag[g], counts[g], "f32")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("counts,K,N", SHAPES, ids=lambda v: str(v)[:24])
def test_grouped_weight_grad(counts, K, N, dtype):
    gen = _gen(4)
    R, E = sum(counts), len(counts)
    x, dy = _randn(gen, R, K, dtype=DT[dtype]), _randn(gen, R, N, dtype=DT[dtype])
    off = offsets_of(counts)
    plan = G.Plan(G.DTYPE_CODES[dtype], G.GEMM_F32)
    for out in ("f32", dtype):
        dw = G.grouped_weight_grad(x, dy, off, alpha=0.5, out_dtype=DT[out], plan=plan)
        assert plan.device_status() == 0
        ref, mag = wgrad_ref(x, dy, off, 0.5)
        check(dw, ref, mag, max(counts), out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("K,N", [(256, 264), (72, 40), (33, 35)])
def test_weight_grad_accumulates_in_place(K, N, out):
    gen = _gen(5)
    counts = [90, 0, 201]
    off = offsets_of(counts)
    x, dy = _randn(gen, 291, K, dtype=DT["bf16"]), _randn(gen, 291, N, dtype=DT["bf16"])
    acc = _randn(gen, 3, K, N, dtype=DT[out])
    ref, mag = wgrad_ref(x, dy, off, 1.0, acc)
    G.grouped_weight_grad(x, dy, off, accumulate=True, out=acc)
    check(acc, ref, mag, 201, out)


@pytest.mark.parametrize("shift", [0, 8, 1])
def test_strided_operands_and_guard_bands(shift):
    """Views into wider buffers (aligned or by one element misaligned), outputs
    inside a buffer whose other entries must stay as they were."""
    gen = _gen(6)
    counts, K, N = [33, 0, 150, 64], 136, 200
    R, off = sum(counts), offsets_of(counts)
    xb, wb = _randn(gen, R, K + 24, dtype=DT["f16"]), _randn(gen, 4, K + 3, N + 32, dtype=DT["f16"])
    dyb = _randn(gen, R, N + 40, dtype=DT["f16"])
    x, w, dy = xb[:, shift:shift + K], wb[:, 1:1 + K, shift:shift + N], dyb[:, shift:shift + N]
    for odt in ("f16", "f32"):
        yb = torch.full((R + 4, N + 24), 3.0, device="cuda", dtype=DT[odt])
        y = yb[2:2 + R, shift:shift + N]
        G.grouped_matmul(x, w, off, out=y)
        check(y, *grouped_ref(x, w, off), K, odt)
        yb[2:2 + R, shift:shift + N] = 3
        assert (yb == 3).all()
        db = torch.full((4, K + 5, N + 16), 3.0, device="cuda", dtype=DT[odt])
        d = db[:, 2:2 + K, shift:shift + N]
        G.grouped_weight_grad(x, dy, off, out=d)
        check(d, *wgrad_ref(x, dy, off), max(counts), odt)
        db[:, 2:2 + K, shift:shift + N] = 3
        assert (db == 3).all()


def test_empty_products():
    off = offsets_of([3, 2])
    x = torch.zeros((5, 0), device="cuda", dtype=DT["bf16"])
    b = torch.tensor([[1.0, -2.0], [3.0, 4.0]], device="cuda")
    y = G.grouped_matmul(x, torch.zeros((2, 0, 2), device="cuda", dtype=DT["bf16"]), off, bias=b, relu=True)
    assert y.tolist() == [[1, 0]] * 3 + [[3, 4]] * 2
    assert G.grouped_matmul(x, torch.zeros((2, 0, 0), device="cuda", dtype=DT["bf16"]), off).shape == (5, 0)
    none = torch.zeros((0, 16), device="cuda", dtype=DT["bf16"])
    dw = G.grouped_weight_grad(none, none, offsets_of([0, 0, 0]))
    assert dw.shape == (3, 16, 16) and (dw == 0).all()


def test_bad_offsets_stay_inside_the_buffer_and_are_reported():
    """Offsets that decrease or leave the buffer are clamped and reported."""
    gen = _gen(7)
    x, w = _randn(gen, 64, 64, dtype=DT["f16"]), _randn(gen, 3, 64, 64, dtype=DT["f16"])
    plan = G.Plan(G.GEMM_F16, G.GEMM_F32)
    buf = torch.full((96, 64), 5.0, device="cuda", dtype=DT["f16"])
    for bad in ([0, 20, 10, 64], [0, 20, 40, 1000], [-5, 10, 20, 64]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        G.grouped_matmul(x, w, off, out=buf[16:80], plan=plan)
        assert plan.device_status() == G.GEMM_ERR_INVALID_ARG
        assert (buf[:16] == 5).all() and (buf[80:] == 5).all()
        G.grouped_weight_grad(x, x, off, plan=plan)
        assert plan.device_status() == G.GEMM_ERR_INVALID_ARG
    G.grouped_matmul(x, w, offsets_of([10, 20, 34]), out=buf[16:80], plan=plan)
    assert plan.device_status() == 0


def test_gradients_are_those_of_the_loss():
    """dX and dW of sum(Y * T) against central differences of the operator
    itself along random directions.  Small integers: every product is exact in
    fp32, so a difference of outputs has no rounding at all."""
    gen = _gen(8)
    counts, K, N = [5, 0, 19, 40], 24, 16
    R, off = sum(counts), offsets_of(counts)
    ints = lambda *s: torch.randint(-3, 4, s, device="cuda", generator=gen)   # noqa: E731
    x, w, t = ints(R, K).to(DT["f16"]), ints(4, K, N).to(DT["f16"]), ints(R, N).to(DT["f16"])
    dx = G.grouped_matmul(t, w.transpose(1, 2), off, out_dtype=DT["f32"])
    dw = G.grouped_weight_grad(x, t, off, out_dtype=DT["f32"])
    loss = lambda x, w: float((G.grouped_matmul(x, w, off, out_dtype=DT["f32"]).double() * t.double()).sum())   # noqa: E731
    for _ in range(3):
        ex, ew = ints(R, K).to(DT["f16"]), ints(4, K, N).to(DT["f16"])
        assert loss(x + ex, w) - loss(x - ex, w) == 2 * float((dx.double() * ex.double()).sum())
        assert loss(x, w + ew) - loss(x, w - ew) == 2 * float((dw.double() * ew.double()).sum())


def test_repeated_calls_agree_bit_for_bit():
    gen = _gen(9)
    counts = [400, 3, 0, 900]
    off = offsets_of(counts)
    x, w = _randn(gen, sum(counts), 512, dtype=DT["bf16"]), _randn(gen, 4, 512, 512, dtype=DT["bf16"])
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    y = G.grouped_matmul(x, w, off, plan=plan, out_dtype=DT["f32"])
    d = G.grouped_weight_grad(x, x, off, plan=plan, out_dtype=DT["f32"])
    for _ in range(4):
        assert torch.equal(y, G.grouped_matmul(x, w, off, plan=plan, out_dtype=DT["f32"]))
        assert torch.equal(d, G.grouped_weight_grad(x, x, off, plan=plan, out_dtype=DT["f32"]))


def test_another_stream():
    gen = _gen(10)
    off = offsets_of([200, 100])
    x, w = _randn(gen, 300, 256, dtype=DT["bf16"]), _randn(gen, 2, 256, 256, dtype=DT["bf16"])
    ref = G.grouped_matmul(x, w, off)
    dref = G.grouped_weight_grad(x, x, off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y, d = G.grouped_matmul(x, w, off), G.grouped_weight_grad(x, x, off)
    s.synchronize()
    assert torch.equal(y, ref) and torch.equal(d, dref)


def test_refusals():
    x = torch.zeros((8, 16), device="cuda", dtype=DT["f16"])
    w = torch.zeros((2, 16, 32), device="cuda", dtype=DT["f16"])
    off = offsets_of([4, 4])
    for bad in (lambda: G.grouped_matmul(x, w[:, :8], off), lambda: G.grouped_matmul(x, w.bfloat16(), off),
                lambda: G.grouped_matmul(x, w, off[:2]), lambda: G.grouped_matmul(x, w, off.long()),
                lambda: G.grouped_matmul(x.t().contiguous().t(), w, off),
                lambda: G.grouped_matmul(x, w, off, out=torch.zeros((8, 31), device="cuda")),
                lambda: G.grouped_matmul(x, w, off, bias=torch.zeros(31, device="cuda")),
                lambda: G.grouped_matmul(x, w.cpu(), off),
                lambda: G.grouped_weight_grad(x, x[:7], off),
                lambda: G.grouped_weight_grad(x, x, off, accumulate=True)):
        with pytest.raises(ValueError):
            bad()

    def code(**kw):
        a = dict(plan=plan.handle, layout_b=G.GEMM_OP_T, groups=2, M=8, N=32, K=16, alpha=1.0, A=x.data_ptr(), lda=16,
                 B=w.data_ptr(), ldb=32, stride_b=512, D=y.data_ptr(), ldd=32, offsets=off.data_ptr())
        a.update(kw)
        with pytest.raises(G.GemmError) as e:
            G.gemm_run_grouped(**a)
        return e.value.status

    y = torch.zeros((8, 32), device="cuda")
    plan = G.Plan(G.GEMM_F16, G.GEMM_F32)
    inv, uns = G.GEMM_ERR_INVALID_ARG, G.GEMM_ERR_UNSUPPORTED
    assert code(groups=-1) == inv and code(lda=15) == inv and code(ldb=31) == inv and code(ldd=31) == inv
    assert code(offsets=None) == inv and code(D=None) == inv and code(layout_b=2) == inv and code(plan=None) == inv
    assert code(groups=1025) == uns and code(M=2 ** 31) == uns
    assert code(epi=G.make_epilogue(G.GEMM_F32, y.data_ptr(), G.GEMM_F32, G.GEMM_BIAS_ROW)) == uns
    assert code(epi=G.make_epilogue(G.GEMM_F32, a_scale=2.0)) == uns
    assert code(epi=G.make_epilogue(G.GEMM_S32)) == inv
    p32 = G.Plan(G.GEMM_F32, G.GEMM_F32)
    assert code(plan=p32.handle) == uns
    with pytest.raises(G.GemmError):   # overlapping outputs
        G.gemm_run_grouped_wgrad(plan.handle, 2, 16, 32, 8, 1.0, x.data_ptr(), 16, x.data_ptr(), 32, 0.0, None, 0, 0,
                                 y.data_ptr(), 32, 16, off.data_ptr(), G.GEMM_F32)
