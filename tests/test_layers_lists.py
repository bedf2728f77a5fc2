"""Lists of tensors: which may share memory.  What is written has its memory to itself, whoever
names the place; what is only read may be listed twice."""
import math

import pytest
import torch

import dense_gemm_epilogues_gb300 as G


def _bad_lists(device):
    a, b, c = (torch.zeros(100, device=device) for _ in range(3))
    return [([a, a], None), ([a, a], [a, a]), ([a, a], [a, c]), ([a, a], [c, a]), ([a, a[:50]], [a, c[:50]]),
            ([a[:50], a], [b[:50], a]), ([a[20:70], a[:50]], [a[20:70], c[:50]]), ([a, b], [c, c]), ([a, b], [c, a])]


@pytest.mark.parametrize("case", range(9))
def test_what_is_written_is_not_shared(case):
    from dense_gemm_epilogues_gb300 import build
    build.build()
    tensors, out = _bad_lists("cpu")[case]
    with pytest.raises(ValueError, match="overlap"):   # (before the device is looked at)
        G.TensorList(tensors, out=out)


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(9))
def test_what_is_written_is_not_shared_on_the_device(case):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tensors, out = _bad_lists("cuda")[case]
    with pytest.raises(ValueError, match="overlap"):
        G.TensorList(tensors, out=out)


@pytest.mark.gpu
def test_lists_partly_in_place():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a, b = (torch.full((n,), 2.0, device="cuda") for n in (1000, 77))
    o = torch.zeros(77, device="cuda")
    norm = G.clip_grad_norm(G.TensorList([a, b], out=[a, o]), 1.0, eps=0.0)
    want = 2 / math.sqrt(4 * 1077)
    assert abs(float(norm) - math.sqrt(4 * 1077)) <= 20 * 2.0 ** -24 * 66
    assert ((a - want).abs() <= 2.0 ** -21).all() and ((o - want).abs() <= 2.0 ** -21).all() and (b == 2).all()


@pytest.mark.gpu
def test_a_norm_of_shared_tensors():
    """Weights that two layers share are counted as often as they are listed; clipping refuses them."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a = torch.full((100,), 2.0, device="cuda")
    for tensors, squares in (([a, a], 800), ([a, a[:50]], 600), ([a.view(10, 10).t(), a], 800)):
        assert abs(float(G.grad_norm(tensors)) - math.sqrt(squares)) <= 20 * 2.0 ** -24 * math.sqrt(squares)
        with pytest.raises(ValueError, match="overlap"):
            G.clip_grad_norm(tensors, 1.0)
    assert (a == 2).all()
    kept = G.TensorList([a])
    assert float(G.grad_norm(kept)) == 20 and float(G.grad_norm(kept)) == 20 and (a == 2).all()
    assert float(G.clip_grad_norm(kept, 1.0, eps=0.0)) == 20 and abs(float(a[0]) - 0.1) < 1e-7
    assert abs(float(G.grad_norm(kept)) - 1) < 1e-6


@pytest.mark.gpu
def test_entries_that_only_count():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a, b = torch.full((1000,), 2.0, device="cuda"), torch.full((77,), 2.0, device="cuda")
    for out in ([None, b], [None, torch.zeros_like(b)], [None, None]):
        b.fill_(2.0)
        assert abs(float(G.clip_grad_norm(G.TensorList([a, b], out=out), 1.0, eps=0.0)) - math.sqrt(4308)) <= 20 * 2.0 ** -24 * 66
        assert (a == 2).all()
        if out[1] is not None:
            assert ((out[1] - 2 / math.sqrt(4308)).abs() <= 2.0 ** -21).all()
    with pytest.raises(ValueError, match="overlap"):
        G.TensorList([a, a], out=[a, None])
    assert abs(float(G.grad_norm(iter([a, b]))) - math.sqrt(4308)) <= 20 * 2.0 ** -24 * 66


@pytest.mark.gpu
def test_a_kept_list_is_laid_out_once():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kept = G.TensorList([torch.ones(10, device="cuda") for _ in range(50)])
    G.grad_norm(kept)
    table = kept.read_table()
    G.grad_norm(kept)
    assert kept.read_table() is table and all(e.dst is None for e in table)
    G.clip_grad_norm(kept, 1e9)
    assert all(e.dst == e.src for e in kept.table)
