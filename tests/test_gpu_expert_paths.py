"""Every variant that the expert-layer operators choose by size, and their use on
other streams and in CUDA graphs.

Which variant ran is read back with Plan.last_config() where it names one."""
import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from expert_helpers import DT, U, check, grouped_ref, newton_schulz_ref, offsets_of, q4_weights, random_q4, wgrad_ref
from test_gpu_orthogonalize import _check, _matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


# Single CTAs; pairs with 64-, 128- and 256-wide tiles of the symmetric products, in one
# block row per matrix (batches) and in several.
@pytest.mark.parametrize("batch,m,n,cta_group", [(3, 130, 140, 1), (20, 200, 800, 2), (30, 130, 140, 2), (80, 130, 140, 2), (120, 130, 140, 2),
                                                 (1, 600, 1500, 1), (1, 1100, 3000, 2), (1, 1700, 1801, 2), (1, 3301, 3400, 2), (1, 3841, 3900, 2)])
@pytest.mark.parametrize("tall", [False, True])
def test_orthogonalize_tiles(batch, m, n, cta_group, tall):
    g = _matrix(batch, m, n, "bf16", 11)
    g = g.transpose(1, 2).contiguous() if tall else g
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    d = G.orthogonalize(g, out_dtype=DT["bf16"], plan=plan)
    assert plan.device_status() == 0 and plan.last_config()["cta_group"] == cta_group
    _check(d, g, "bf16")


@pytest.mark.parametrize("counts,K,N,cta_group", [([100, 0, 200], 200, 264, 1), ([123], 64, 20000, 1), ([300], 72, 4096, 1),
                                                  ([500, 0, 13, 257], 200, 4101, 2), ([600], 72, 12000, 2),
                                                  ([128, 1, 255, 128], 64, 5000, 2)], ids=str)
@pytest.mark.parametrize("layout", ["N", "K"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_grouped_tiles(counts, K, N, cta_group, layout, dtype):
    gen = _gen(1)
    R, E = sum(counts), len(counts)
    off = offsets_of(counts, 3)
    x = torch.randn((R + 4, K), device="cuda", generator=gen).to(DT[dtype])
    x[:3] = float("nan")
    w = torch.randn((E, K, N), device="cuda", generator=gen).to(DT[dtype])
    if layout == "K":
        w = w.transpose(1, 2).contiguous().transpose(1, 2)
    b = torch.randn((E, N), device="cuda", generator=gen)
    plan = G.Plan(G.DTYPE_CODES[dtype], G.GEMM_F32)
    y = torch.full((R + 4, N), 5.0, device="cuda", dtype=DT[dtype])
    G.grouped_matmul(x, w, off, bias=b, relu=True, out=y, plan=plan)
    assert plan.last_config()["cta_group"] == cta_group and plan.device_status() == 0
    ref, mag = grouped_ref(x, w, off, b, True)
    check(y[3:-1], ref[3:-1], mag[3:-1], K, dtype)
    assert (y[:3] == 5).all() and (y[-1] == 5).all()


@pytest.mark.parametrize("counts,cta_group", [([700, 3, 300], 2), ([256], 2), ([2000, 0, 0, 1], 2), ([251], 1), ([90, 0, 300], 1)],
                         ids=str)
@pytest.mark.parametrize("K,N", [(200, 264), (130, 1000), (129, 131)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_weight_gradient_tiles(counts, cta_group, K, N, out):
    gen = _gen(6)
    R, E = sum(counts), len(counts)
    off = offsets_of(counts, 3)
    x = torch.randn((R + 4, K), device="cuda", generator=gen).bfloat16()
    dy = torch.randn((R + 4, N), device="cuda", generator=gen).bfloat16()
    for t in (x, dy):
        t[:3] = float("nan")
        t[-1] = float("inf")
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    dw = G.grouped_weight_grad(x, dy, off, out_dtype=DT[out], plan=plan)
    assert plan.last_config()["cta_group"] == cta_group and plan.device_status() == 0
    check(dw, *wgrad_ref(x, dy, off), max(counts), out)


# Decoded inside the product in one, two and four passes, and decoded once for the
# tensor-core kernel on single CTAs and on pairs; experts with uneven rows.
@pytest.mark.parametrize("counts,K,N", [([32], 512, 2048), ([64], 2048, 1024), ([128], 4096, 512), ([100], 512, 20000),
                                        ([300], 256, 4096), ([5, 200, 0, 90], 256, 1000), ([0, 0, 256], 512, 4000)], ids=str)
@pytest.mark.parametrize("sdt", ["f32", "bf16"])
def test_q4_paths(counts, K, N, sdt):
    gen = _gen(2)
    R, E = sum(counts), len(counts)
    x = torch.randn((R, K), device="cuda", generator=gen).bfloat16()
    q, s, z = random_q4(N, K, 64, DT[sdt], True, gen, E)
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    off = offsets_of(counts)
    y = G.q4_matmul(x, q, s, 64, zeros=z, offsets=off, out_dtype=DT["f32"], plan=plan)
    assert plan.device_status() == 0
    w, o = q4_weights(q, s, z, K, 64), off.tolist()
    for g in range(E):
        r = slice(o[g], o[g + 1])
        v = w[g].double()
        check(y[r], x[r].double() @ v.mT, x[r].double().abs() @ v.mT.abs(), K, "f32", U["bf16"] if R > 32 else 0.0)


@pytest.mark.parametrize("rank", [1, 30, 100])
def test_orthogonalize_of_gradients_of_few_rows(rank):
    """A weight gradient of `rank` rows has so many singular values.  In the directions that
    it lacks, the rounding of X to fp16 before step k (relative 2^-11) grows by a in every
    later step, and nothing in the exact result is there to hide it: at most
    2^-11 * sum over k of a^(5 - k) |X_k|, |X_k| <= min(a^k, 1.21 sqrt(rank)) (a singular
    value grows by at most a per step and is at most 1.21 once it has come near one)."""
    a = 3.4445
    noise = 2.0 ** -11 * sum(a ** (5 - k) * min(a ** k, 1.21 * rank ** 0.5) for k in range(5))
    gen = _gen(4)
    g = torch.randn((192, rank), device="cuda", generator=gen) @ torch.randn((rank, 256), device="cuda", generator=gen)
    d, ref = G.orthogonalize(g, out_dtype=DT["f32"]).double(), newton_schulz_ref(g)
    assert (d - ref).norm() <= noise + 3.5e-3 * ref.norm()


def test_other_streams_and_graphs():
    """Work queued on a side stream behind the inputs' making; then a captured graph of all
    operators, replayed on new values in the same buffers."""
    gen = _gen(3)
    E, R, K, N = 4, 150, 192, 256
    off = offsets_of([30, 70, 0, 50])
    x = torch.empty((R, K), device="cuda", dtype=DT["bf16"])
    dy = torch.empty((R, N), device="cuda", dtype=DT["bf16"])
    w = torch.randn((E, K, N), device="cuda", generator=gen).bfloat16()
    q, s, z = random_q4(N, K, 64, DT["bf16"], True, gen, E)
    qw = q4_weights(q, s, z, K, 64)
    plan, plan32 = G.Plan(G.GEMM_BF16, G.GEMM_F32), G.Plan(G.GEMM_F32, G.GEMM_F32)

    def step():
        y = G.grouped_matmul(x, w, off, out_dtype=DT["f32"], plan=plan)
        dw = G.grouped_weight_grad(x, dy, off, out_dtype=DT["f32"], plan=plan)
        return y, dw, G.q4_matmul(x, q, s, 64, zeros=z, offsets=off, out_dtype=DT["f32"], plan=plan), \
            G.orthogonalize(dw, plan=plan32)

    def fill(seed):
        x.copy_(torch.randn((R, K), device="cuda", generator=_gen(seed)))
        dy.copy_(torch.randn((R, N), device="cuda", generator=_gen(seed + 1)))

    def verify(y, dw, y4, up):
        check(y, *grouped_ref(x, w, off), K, "f32")
        check(dw, *wgrad_ref(x, dy, off), R, "f32")
        check(y4, *grouped_ref(x, qw.mT, off), K, "f32", U["bf16"])
        assert (up[2] == 0).all() and torch.equal(up, G.orthogonalize(dw, plan=plan32))
        assert plan.device_status() == 0 and plan32.device_status() == 0

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fill(5)
        out = step()
    side.synchronize()
    verify(*out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (7, 9):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        verify(*out)
