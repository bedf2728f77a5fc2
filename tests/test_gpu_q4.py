"""Products with 4-bit weights (gemm_run_q4) against a plain 64-bit form: one
token to a prompt, odd sizes, every group size and type, zero points, experts,
strided and misaligned operands."""
import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from expert_helpers import DT, U, check, offsets_of, q4_weights, random_q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _ref(x, w, bias=None, relu=False, alpha=1.0):
    ref, mag = alpha * (x.double() @ w.mT), abs(alpha) * (x.double().abs() @ w.mT.abs())
    if bias is not None:
        ref, mag = ref + bias.double(), mag + bias.double().abs()
    return (ref.clamp(min=0) if relu else ref), mag


# Prompts may round each weight to the operands' 16-bit type on its way to the tensor
# cores; a few tokens never do.
FEW = 32


def _extra(rows, dtype):
    return U[dtype] if rows > FEW else 0.0


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 3, 7, 8, 9, 16, 17, 31, 32, 33, 64, 100, 257])
@pytest.mark.parametrize("N,K,group", [(64, 64, 32), (200, 512, 128), (33, 1056, 32), (1, 32, 32), (500, 2048, 64)])
def test_q4_dense(N, K, group, rows, dtype, zeros):
    gen = _gen(1)
    x = torch.randn((rows, K), device="cuda", generator=gen).to(DT[dtype])
    q, s, z = random_q4(N, K, group, DT[dtype], zeros, gen)
    w = q4_weights(q, s, z, K, group)
    plan = G.Plan(G.DTYPE_CODES[dtype], G.GEMM_F32)
    for out in ("f32", dtype):
        y = G.q4_matmul(x, q, s, group, zeros=z, out_dtype=DT[out], plan=plan)
        check(y, *_ref(x, w), K, out, _extra(rows, dtype))
    assert plan.device_status() == 0


@pytest.mark.parametrize("sdt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K,group", [(1, 32), (31, 32), (33, 32), (95, 64), (100, 96), (4095, 128), (416, 416), (70, 4096)])
@pytest.mark.parametrize("rows", [1, 5, 40])
def test_q4_odd_depths_and_groups(K, group, rows, sdt):
    gen = _gen(2)
    x = torch.randn((rows, K), device="cuda", generator=gen).to(DT["bf16"])
    q, s, z = random_q4(77, K, group, DT[sdt], True, gen)
    y = G.q4_matmul(x, q, s, group, zeros=z, out_dtype=DT["f32"])
    check(y, *_ref(x, q4_weights(q, s, z, K, group)), K, "f32", _extra(rows, "bf16"))


@pytest.mark.parametrize("counts", [[1], [0, 1, 0], [3, 0, 1, 8, 9], [0, 40, 2], [17, 33, 64, 1], [300, 5, 0, 90]],
                         ids=str)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_q4_experts(counts, dtype):
    gen = _gen(3)
    E, R, N, K, group = len(counts), sum(counts), 136, 320, 64
    off = offsets_of(counts, 2)
    x = torch.randn((R + 5, K), device="cuda", generator=gen).to(DT[dtype])
    x[:2] = float("nan")
    q, s, z = random_q4(N, K, group, DT["f32"], True, gen, E)
    b = torch.randn((E, N), device="cuda", generator=gen)
    out = torch.full((R + 5, N), 9.0, device="cuda")
    G.q4_matmul(x, q, s, group, zeros=z, offsets=off, alpha=0.5, bias=b, relu=True, out=out)
    o = off.tolist()
    w = q4_weights(q, s, z, K, group)
    for g in range(E):
        r = slice(o[g], o[g + 1])
        check(out[r], *_ref(x[r], w[g], b[g], True, 0.5), K, "f32", _extra(R, dtype))
    assert (out[:2] == 9).all() and (out[2 + R:] == 9).all()


@pytest.mark.parametrize("rows", [1, 6, 50])
@pytest.mark.parametrize("shift", [0, 16, 1])
def test_q4_strided_operands_and_guard_bands(rows, shift):
    gen = _gen(4)
    N, K, group = 90, 256, 32
    xb = torch.randn((rows, K + 32), device="cuda", generator=gen).half()
    q, s, z = random_q4(N, K + 64, group, DT["f16"], True, gen)
    x, q, s, z = xb[:, shift:shift + K], q[:, shift:shift + K // 2], s[:, :K // group], z[:, :K // group]
    yb = torch.full((rows + 2, N + 24), 3.0, device="cuda", dtype=DT["f16"])
    y = yb[1:1 + rows, shift:shift + N][:, :N]
    n = y.shape[1]
    G.q4_matmul(x, q[:n], s[:n], group, zeros=z[:n], out=y)
    check(y, *_ref(x, q4_weights(q, s, z, K, group)[:n]), K, "f16", _extra(rows, "f16"))
    yb[1:1 + rows, shift:shift + n] = 3
    assert (yb == 3).all()


@pytest.mark.parametrize("rows", [1, 4, 40])
def test_q4_infinities_stay_in_their_rows(rows):
    gen = _gen(5)
    x = torch.randn((rows + 2, 128), device="cuda", generator=gen).half()
    x[1, 5], x[0, 7] = float("inf"), float("nan")
    q, s, _ = random_q4(48, 128, 32, DT["f16"], False, gen)
    y = G.q4_matmul(x, q, s, 32, out_dtype=DT["f32"])
    assert y[0].isnan().all() and not y[1].isfinite().any()
    check(y[2:], *_ref(x[2:], q4_weights(q, s, None, 128, 32)), 128, "f32", _extra(rows + 2, "f16"))


@pytest.mark.parametrize("zero_points", [False, True])
def test_quantize_q4_is_the_nearest_grid_point(zero_points):
    """Every value is within half a step (plus the scale's own rounding) of its
    weight, also for groups that are all zero."""
    gen = _gen(6)
    w = torch.randn((40, 256), device="cuda", generator=gen)
    w[3, :64] = 0
    q, s, z = G.quantize_q4(w, 64, zero_points=zero_points)
    back = q4_weights(q, s, z, 256, 64)
    step = s.double().repeat_interleave(64, 1)
    assert ((back - w.double()).abs() <= step * (0.5 + (0.5 if zero_points else 0) + 1e-5)).all()
    assert (back[3, :64] == 0).all()
    x = torch.randn((3, 256), device="cuda", generator=gen).half()
    check(G.q4_matmul(x, q, s, 64, zeros=z, out_dtype=DT["f32"]), *_ref(x, back), 256, "f32")


def test_q4_empty_and_refusals():
    gen = _gen(7)
    x = torch.randn((4, 64), device="cuda", generator=gen).half()
    q, s, z = random_q4(32, 64, 32, DT["f16"], True, gen)
    assert G.q4_matmul(x[:0], q, s, 32).shape == (0, 32)
    assert G.q4_matmul(x, q[:0], s[:0], 32).shape == (4, 0)
    b = torch.arange(32, device="cuda", dtype=torch.float32)
    assert torch.equal(G.q4_matmul(x[:, :0], q[:, :0], s[:, :0], 32, bias=b, out_dtype=DT["f32"]), b.expand(4, 32))
    for bad in (lambda: G.q4_matmul(x, q, s, 48), lambda: G.q4_matmul(x, q, s, 64), lambda: G.q4_matmul(x, q.int(), s, 32),
                lambda: G.q4_matmul(x[:, :60], q, s, 32), lambda: G.q4_matmul(x, q, s, 32, zeros=z.int()),
                lambda: G.q4_matmul(x, torch.stack([q, q]), torch.stack([s, s]), 32),
                lambda: G.q4_matmul(x, q, s, 32, out=torch.zeros((4, 31), device="cuda")),
                lambda: G.quantize_q4(torch.zeros((4, 100), device="cuda"), 32)):
        with pytest.raises(ValueError):
            bad()
    y = torch.zeros((4, 32), device="cuda")
    p32 = G.Plan(G.GEMM_F32, G.GEMM_F32)
    with pytest.raises(G.GemmError) as e:
        G.q4_matmul(x, q, s, 32, plan=p32)
    assert e.value.status == G.GEMM_ERR_UNSUPPORTED
    plan = G.Plan(G.GEMM_F16, G.GEMM_F32)

    def code(groups=1, offsets=None, K=64, ldd=32, **kw):
        f = dict(values=q.data_ptr(), ld_values=32, scales=s.data_ptr(), scale_dtype=G.GEMM_F16, ld_scales=2,
                 group_size=32)
        f.update(kw)
        with pytest.raises(G.GemmError) as e:
            G.gemm_run_q4(plan.handle, groups, 4, 32, K, 1.0, x.data_ptr(), 64, G.gemm_q4_t(**f), y.data_ptr(), ldd,
                          offsets)
        return e.value.status

    for kw in (dict(groups=2), dict(ldd=31), dict(ld_values=31), dict(ld_scales=1), dict(group_size=33),
               dict(group_size=0), dict(scale_dtype=G.GEMM_S8), dict(values=None), dict(scales=None),
               dict(zeros=z.data_ptr(), ld_zeros=1), dict(stride_values=-1)):
        assert code(**kw) == G.GEMM_ERR_INVALID_ARG, kw


def test_a_plan_of_another_type_is_refused():
    gen = _gen(8)
    q, s, _ = random_q4(32, 64, 32, DT["f16"], False, gen)
    x = torch.randn((4, 64), device="cuda", generator=gen).half()
    w = torch.zeros((1, 64, 32), device="cuda", dtype=DT["f16"])
    off = offsets_of([4])
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    for call in (lambda: G.q4_matmul(x, q, s, 32, plan=plan), lambda: G.grouped_matmul(x, w, off, plan=plan),
                 lambda: G.grouped_weight_grad(x, x, off, plan=plan), lambda: G.orthogonalize(x, plan=plan)):
        with pytest.raises(G.GemmError) as e:
            call()
        assert e.value.status == G.GEMM_ERR_UNSUPPORTED
