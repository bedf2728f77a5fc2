"""Which variant of an expert-layer operator a size runs, read back with Plan.last_config(),
and its results: exact weights wherever the 4-bit product decodes inside, whatever the number
of rows."""
import os
import subprocess
import sys

import pytest
import torch

import dense_gemm_epilogues_gb300 as G
from expert_helpers import DT, U, check, offsets_of, q4_weights, random_q4
from test_gpu_orthogonalize import _check, _matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_library()


INSIDE = [  # rows of each expert, K, N, rows per pass, columns per CTA: more than, at most
    ([1], 512, 4096, 8, 0, 16), ([1], 256, 7296, 8, 16, 32), ([1], 512, 20000, 8, 32, 48),
    ([5, 0, 3], 256, 3000, 8, 16, 32), ([12], 512, 2048, 16, 0, 32), ([0, 40, 2], 256, 1000, 16, 0, 32),
    ([32], 512, 2048, 32, 0, 32), ([64], 2048, 1024, 32, 0, 32), ([128], 4096, 512, 32, 0, 32)]
ONCE = [([100], 512, 20000, 1), ([300], 256, 4096, 1), ([5, 200, 0, 90], 256, 1000, 1), ([0, 0, 256], 512, 4000, 1),
        ([600], 256, 12000, 2)]


def _q4(counts, K, N, sdt, dtype="bf16"):
    gen = torch.Generator("cuda").manual_seed(2)
    E = len(counts)
    x = torch.randn((sum(counts), K), device="cuda", generator=gen).to(DT[dtype])
    q, s, z = random_q4(N, K, 64, DT[sdt], True, gen, E)
    plan, off = G.Plan(G.DTYPE_CODES[dtype], G.GEMM_F32), offsets_of(counts)
    y = G.q4_matmul(x, q, s, 64, zeros=z, offsets=off, out_dtype=DT["f32"], plan=plan)
    assert plan.device_status() == 0
    w, o = q4_weights(q, s, z, K, 64), off.tolist()
    parts = [(slice(o[g], o[g + 1]), w[g]) for g in range(E)]
    ref = torch.cat([x[r].double() @ v.mT for r, v in parts])
    mag = torch.cat([x[r].double().abs() @ v.abs().mT for r, v in parts])
    return y, ref, mag, plan.last_config()


@pytest.mark.parametrize("counts,K,N,rows,above,most", INSIDE, ids=str)
@pytest.mark.parametrize("sdt", ["f32", "bf16"])
def test_4_bit_inside(counts, K, N, rows, above, most, sdt):
    y, ref, mag, cfg = _q4(counts, K, N, sdt)
    assert cfg["kernel"] == G.GEMM_KERNEL_SIMT and cfg["bm"] == rows and above < cfg["bn"] <= most
    check(y, ref, mag, K, "f32")


@pytest.mark.parametrize("counts,K,N,cta_group", ONCE, ids=str)
@pytest.mark.parametrize("sdt", ["f32", "bf16"])
def test_4_bit_once(counts, K, N, cta_group, sdt):
    y, ref, mag, cfg = _q4(counts, K, N, sdt)
    assert cfg["kernel"] == (G.GEMM_KERNEL_TC, G.GEMM_KERNEL_TC_PAIR)[cta_group - 1] and cfg["cta_group"] == cta_group
    check(y, ref, mag, K, "f32", U["bf16"])


# Tiles of the symmetric products 64, 128 and 256 wide.
@pytest.mark.parametrize("batch,m,n,cta_group,width", [
    (3, 130, 140, 1, 64), (1, 600, 1500, 1, 64), (20, 200, 800, 2, 64), (1, 1100, 3000, 2, 64), (30, 130, 140, 2, 128),
    (1, 1700, 1801, 2, 128), (120, 130, 140, 2, 256), (1, 3841, 3900, 2, 256)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_orthogonalize_widths(batch, m, n, cta_group, width, out):
    g = _matrix(batch, m, n, "bf16", 11)
    plan = G.Plan(G.GEMM_BF16, G.GEMM_F32)
    d = G.orthogonalize(g, out_dtype=DT[out], plan=plan)
    cfg = plan.last_config()
    assert plan.device_status() == 0 and cfg["cta_group"] == cta_group and cfg["bn"] == width
    _check(d, g, out)


def test_calls_without_a_product_say_so():
    plan = G.Plan(G.GEMM_F32, G.GEMM_F32)
    g = torch.ones((8, 12), device="cuda")
    G.orthogonalize(g, plan=plan)
    assert plan.last_config()["kernel"] == G.GEMM_KERNEL_TC
    G.orthogonalize(g, steps=0, plan=plan)
    assert plan.last_config()["kernel"] == G.GEMM_KERNEL_NONE
    G.orthogonalize(g, plan=plan)
    G.orthogonalize(g[:0], plan=plan)
    assert plan.last_config()["kernel"] == G.GEMM_KERNEL_NONE


def test_every_launch_is_logged():
    """GEMM_LOG=1 prints one line per call, 4-bit products of a few rows included."""
    code = ("import torch, dense_gemm_epilogues_gb300 as G\n"
            "x = torch.ones((3, 64), device='cuda', dtype=torch.float16)\n"
            "q = torch.zeros((40, 32), device='cuda', dtype=torch.uint8)\n"
            "G.q4_matmul(x, q, torch.ones((40, 1), device='cuda'), 64)\n"
            "torch.cuda.synchronize()\n")
    env = dict(os.environ, GEMM_LOG="1")
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "gemm: q4 M=3 N=40 K=64" in r.stderr, r.stderr
