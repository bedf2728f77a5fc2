"""Lists of tensors: which may share memory.  What is written has its memory to itself, whoever
names the place."""
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
