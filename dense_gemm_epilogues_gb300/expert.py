"""Expert layers on torch tensors: products grouped by expert and their weight
gradient, products with 4-bit weights, orthogonalised updates.

The functions check their arguments, read pointers, strides and the current
stream and call the C entry points of include/gemm.h; a decoding step calls them
once per layer and matrix, so they are written to take little host time.

A call without `plan` uses one that is kept for its thread, stream and operand type,
so it waits for nothing; default_plan_status() reports errors found on the device.  Such
plans keep their scratch: a program that wants it back, that runs captured graphs at the
same time (a capture's stream gives its graphs one plan), or that reads the status of
single calls makes its own.  Nothing is recorded for autograd.
"""
from __future__ import annotations

import ctypes
import threading
from typing import Optional

import torch

from . import (GEMM_ACT_NONE, GEMM_ACT_RELU, GEMM_BF16, GEMM_BIAS_COL, GEMM_BIAS_NONE, GEMM_ERR_UNSUPPORTED, GEMM_F16,
               GEMM_F32, GEMM_OP_N, GEMM_OP_T, GemmError, Plan, gemm_epilogue_t, gemm_q4_t, load_library)

_CODES = {torch.float32: GEMM_F32, torch.float16: GEMM_F16, torch.bfloat16: GEMM_BF16}
_LIB = load_library()
_raw_stream = torch._C._cuda_getCurrentRawStream


def _code(dtype) -> int:
    try:
        return _CODES[dtype]
    except KeyError:
        raise ValueError(f"type {dtype} is not float32, float16 or bfloat16") from None


# The epilogues without a bias, by (ReLU, output type): they hold no pointer.
_PLAIN = {(relu, code): gemm_epilogue_t(None, GEMM_F32, GEMM_BIAS_NONE, GEMM_ACT_RELU if relu else GEMM_ACT_NONE, code,
                                        GEMM_ACT_NONE, 1.0)
          for relu in (False, True) for code in _CODES.values()}


def _device(x, *others) -> int:
    """The CUDA device that all tensors are on."""
    d = x.get_device()
    if d < 0:
        raise ValueError("tensors must be on a CUDA device")
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError("tensors are on different devices")
    return d


# The plans of calls that are given none: per thread by (device, stream, operand type,
# c_dtype), so calls that can overlap never share scratch.  A thread that ends leaves its
# plans to later ones on the same streams; none is destroyed (a captured graph may use it).
_DEFAULTS = []   # all of them
_FREE = {}       # lists of those whose thread has ended


class _Lease(dict):
    def __del__(self, free=_FREE):   # (bound here: at exit the module's names may be gone)
        for key, plan in self.items():
            free.setdefault(key, []).append(plan)


class _Thread(threading.local):
    def __init__(self):
        self.plans = _Lease()


_THREAD = _Thread()


def _default_plan(key) -> Plan:
    try:
        plan = _FREE[key].pop()
    except (KeyError, IndexError):
        device, _, ab_code, c_code = key
        plan = Plan(ab_code, c_code, device)
        _DEFAULTS.append(plan)
    _THREAD.plans[key] = plan
    return plan


def _plan_for(plan, ab_code: int, c_code: int, device: int, stream: int) -> Plan:
    """The caller's plan, which has to be for these operands, or this stream's default one."""
    if plan is None:
        key = (device, stream, ab_code, c_code)
        return _THREAD.plans.get(key) or _default_plan(key)
    if plan.ab_dtype != ab_code:
        raise GemmError(GEMM_ERR_UNSUPPORTED, "a plan of another operand type")
    if plan.device != device:
        raise ValueError("the plan is on another device")
    return plan


def default_plan_status(device=None) -> int:
    """What gemm_plan_device_status reports of calls that were given no plan: the first error
    (GEMM_ERR_INVALID_ARG for bad offsets, GEMM_ERR_TIMEOUT for an expired wait) of all
    threads and streams since the last time, or 0.  Waits for the device (the current one, or
    `device`) and clears what it reports; not during a stream capture."""
    index = torch.cuda.current_device() if device is None else torch.device(device).index or 0
    torch.cuda.synchronize(index)
    code = 0
    for plan in list(_DEFAULTS):
        if plan.device == index:
            code = plan.device_status() or code
    return code


def _pitch(shape, stride, name: str) -> int:
    """Leading dimension of a row-major 2-D view."""
    rows, cols = shape
    if (stride[1] != 1 and cols > 1) or (rows > 1 and stride[0] < cols):
        raise ValueError(f"{name} must be row-major")
    return max(stride[0], cols, 1)


def _check_offsets(offsets, groups: int):
    if offsets.dtype is not torch.int32 or offsets.shape != (groups + 1,) or offsets.stride() != (1,):
        raise ValueError("offsets must be a contiguous int32 tensor of groups + 1 entries")


def _epilogue(bias, groups: int, n: int, relu: bool, out_code: int):
    """(epilogue, bias stride) of a grouped product; bias is [groups, N] or [N] (shared)."""
    if bias is None:
        return _PLAIN[bool(relu), out_code], 0
    act = GEMM_ACT_RELU if relu else GEMM_ACT_NONE
    if bias.shape not in ((groups, n), (n,)) or (bias.stride(-1) != 1 and n > 1):
        raise ValueError("bias must be [N] or [groups, N] with contiguous rows")
    return (gemm_epilogue_t(bias.data_ptr(), _code(bias.dtype), GEMM_BIAS_COL, act, out_code, GEMM_ACT_NONE, 1.0),
            bias.stride(0) if bias.dim() == 2 else 0)


def _output(out, M: int, N: int, dtype, like):
    """(out, its pitch, its type code): a new [M, N] tensor, or the caller's."""
    if out is None:
        return torch.empty((M, N), dtype=dtype, device=like.device), max(N, 1), _code(dtype)
    if out.shape != (M, N):
        raise ValueError("out must be [rows, N]")
    return out, _pitch((M, N), out.stride(), "out"), _code(out.dtype)


def grouped_matmul(x, w, offsets, *, alpha: float = 1.0, bias=None, relu: bool = False, out=None, out_dtype=None,
                   plan: Optional[Plan] = None, stream=None):
    """out[r] = act(alpha * x[r] @ w[g] + bias[g]) for the rows r of each group g
    (gemm_run_grouped): the forward product of an expert layer, and with
    w.transpose(1, 2) its input gradient.

    x: [rows, K] float16 or bfloat16, rows sorted by group; w: [groups, K, N]
    with unit stride along K or N; offsets: int32 [groups + 1] on the device,
    group g owning rows offsets[g] .. offsets[g + 1] - 1 (rows of no group are
    left as they are in `out`).  bias: [groups, N] or [N].  out_dtype defaults
    to x's.  Returns `out`."""
    dtype = x.dtype
    M, K = x.shape
    groups, K2, N = w.shape
    if K2 != K or w.dtype is not dtype:
        raise ValueError("x must be [rows, K] and w [groups, K, N] of the same type")
    _check_offsets(offsets, groups)
    device = _device(x, w, offsets, bias, out)
    lda = _pitch((M, K), x.stride(), "x")
    ws, wk, wn = w.stride()
    if (wn == 1 or N <= 1) and (wk >= N or K <= 1):
        lb, ldb = GEMM_OP_T, max(wk, N, 1)
    elif (wk == 1 or K <= 1) and (wn >= K or N <= 1):
        lb, ldb = GEMM_OP_N, max(wn, K, 1)
    else:
        raise ValueError("w must have unit stride along K or N and no overlapping rows")
    out, ldd, code = _output(out, M, N, out_dtype or dtype, x)
    stream = _raw_stream(device) if stream is None else stream
    plan = _plan_for(plan, _code(dtype), GEMM_F32, device, stream)
    epi, stride_bias = _epilogue(bias, groups, N, relu, code)
    status = _LIB.gemm_run_grouped(plan.handle, lb, groups, M, N, K, alpha, x.data_ptr(), lda, w.data_ptr(), ldb,
                                   ws if groups > 1 else 0, out.data_ptr(), ldd, offsets.data_ptr(), epi, stride_bias,
                                   stream)
    if status:
        raise GemmError(status, "gemm_run_grouped")
    return out


def grouped_weight_grad(x, dy, offsets, *, alpha: float = 1.0, accumulate: bool = False, out=None, out_dtype=None,
                        plan: Optional[Plan] = None, stream=None):
    """out[g] = alpha * x[rows of g].T @ dy[rows of g] (+ out[g] if accumulate): the
    weight gradient of grouped_matmul (gemm_run_grouped_wgrad); an empty group
    gives zeros.

    x: [rows, K], dy: [rows, N], float16 or bfloat16; offsets as for
    grouped_matmul.  out: [groups, K, N] with contiguous rows; accumulate needs
    `out` and a plan whose c_dtype is out's type (made here if none is given).
    out_dtype defaults to x's.  Returns `out`."""
    dtype = x.dtype
    rows, M = x.shape
    rows2, N = dy.shape
    if rows2 != rows or dy.dtype is not dtype:
        raise ValueError("x must be [rows, K] and dy [rows, N] of the same type")
    groups = offsets.shape[0] - 1
    _check_offsets(offsets, groups)
    device = _device(x, dy, offsets, out)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((groups, M, N), dtype=out_dtype or dtype, device=x.device)
    elif out.shape != (groups, M, N) or (out.stride(2) != 1 and N > 1) or (out.stride(1) < N and M > 1):
        raise ValueError("out must be [groups, K, N] with contiguous rows")
    code = _code(out.dtype)
    stream = _raw_stream(device) if stream is None else stream
    plan = _plan_for(plan, _code(dtype), code if accumulate else GEMM_F32, device, stream)
    if accumulate and plan.c_dtype != code:
        raise ValueError("accumulate needs a plan whose c_dtype is out's type")
    ldd = max(out.stride(1), N, 1)
    stride_d = out.stride(0) if groups > 1 else M * ldd
    p = out.data_ptr()
    status = _LIB.gemm_run_grouped_wgrad(plan.handle, groups, M, N, rows, alpha, x.data_ptr(),
                                         _pitch((rows, M), x.stride(), "x"), dy.data_ptr(),
                                         _pitch((rows, N), dy.stride(), "dy"), 1.0 if accumulate else 0.0,
                                         p if accumulate else None, ldd, stride_d, p, ldd, stride_d,
                                         offsets.data_ptr(), code, stream)
    if status:
        raise GemmError(status, "gemm_run_grouped_wgrad")
    return out


def quantize_q4(w, group_size: int, *, zero_points: bool = False, scale_dtype=None):
    """Round-to-nearest 4-bit weights for q4_matmul: (q, scales, zeros) of w
    [..., N, K] (K a multiple of group_size), zeros None unless zero_points.  One
    scale per row and group_size entries of K; done once per weight matrix."""
    if group_size <= 0 or group_size % 32 or w.shape[-1] % group_size:
        raise ValueError("group_size must be a multiple of 32 that divides K")
    scale_dtype = scale_dtype or w.dtype
    g = w.float().unflatten(-1, (-1, group_size))
    if zero_points:
        lo, hi = g.amin(-1).clamp(max=0), g.amax(-1).clamp(min=0)
        scales = ((hi - lo) / 15).to(scale_dtype)
    else:
        scales = (g.abs().amax(-1) / 7).to(scale_dtype)
    div = torch.where(scales == 0, 1.0, scales.float())[..., None]
    zeros = torch.round(-lo[..., None] / div).clamp(0, 15) if zero_points else torch.full_like(div, 8)
    v = (torch.round(g / div) + zeros).clamp(0, 15).flatten(-2).to(torch.uint8)
    return v[..., 0::2] | (v[..., 1::2] << 4), scales, zeros[..., 0].to(torch.uint8) if zero_points else None


def q4_matmul(x, q, scales, group_size: int, *, zeros=None, offsets=None, alpha: float = 1.0, bias=None,
              relu: bool = False, out=None, out_dtype=None, plan: Optional[Plan] = None, stream=None):
    """out = act(alpha * x @ w.T + bias) with 4-bit weights (gemm_run_q4):
    w[n, k] = scales[n, k // group_size] * (q[n, k] - zeros[n, k // group_size]).

    x: [rows, K] float16 or bfloat16; q: uint8 [N, ceil(K / 2)], two weights a
    byte, the even k in the low half; scales: [N, ceil(K / group_size)] of a
    floating type; zeros: uint8 like scales, or None for 8.  Experts' weights have
    a leading dimension [groups], and `offsets` gives every group's rows as for
    grouped_matmul (without it, one group of all rows).  bias: [N] or [groups, N].
    Returns `out`."""
    dtype = x.dtype
    M, K = x.shape
    shape = q.shape
    groups = shape[0] if len(shape) == 3 else 1
    if len(shape) not in (2, 3) or q.dtype is not torch.uint8:
        raise ValueError("q must be uint8 [N, K / 2] or [groups, N, K / 2]")
    N = shape[-2]
    if group_size <= 0 or group_size % 32:
        raise ValueError("group_size must be a positive multiple of 32")
    kg = -(-K // group_size)
    want = shape[:-1] + (kg,)
    if shape[-1] != (K + 1) // 2 or scales.shape != want or \
            (zeros is not None and (zeros.shape != want or zeros.dtype is not torch.uint8)):
        raise ValueError("q, scales or zeros do not match x and group_size")
    if offsets is not None:
        _check_offsets(offsets, groups)
    elif groups != 1:
        raise ValueError("experts' weights need offsets")
    device = _device(x, q, scales, zeros, offsets, bias, out)
    qs, ss, zs = q.stride(), scales.stride(), zeros.stride() if zeros is not None else None
    if (qs[-1] != 1 and shape[-1] > 1) or (kg > 1 and (ss[-1] != 1 or (zs is not None and zs[-1] != 1))) or \
            (N > 1 and (qs[-2] < shape[-1] or ss[-2] < kg or (zs is not None and zs[-2] < kg))):
        raise ValueError("q, scales and zeros need contiguous rows that do not overlap")
    out, ldd, code = _output(out, M, N, out_dtype or dtype, x)
    stream = _raw_stream(device) if stream is None else stream
    plan = _plan_for(plan, _code(dtype), GEMM_F32, device, stream)
    epi, stride_bias = _epilogue(bias, groups, N, relu, code)
    ex = groups > 1
    weights = gemm_q4_t(q.data_ptr(), max(qs[-2], shape[-1]), qs[0] if ex else 0, scales.data_ptr(),
                        _code(scales.dtype), max(ss[-2], kg), ss[0] if ex else 0,
                        zeros.data_ptr() if zeros is not None else None, max(zs[-2], kg) if zs is not None else 0,
                        zs[0] if ex and zs is not None else 0, group_size)
    status = _LIB.gemm_run_q4(plan.handle, groups, M, N, K, alpha, x.data_ptr(), _pitch((M, K), x.stride(), "x"),
                              weights, out.data_ptr(), ldd, offsets.data_ptr() if offsets is not None else None, epi,
                              stride_bias, stream)
    if status:
        raise GemmError(status, "gemm_run_q4")
    return out


def orthogonalize(g, *, steps: int = 5, coeffs=(3.4445, -4.7750, 2.0315), eps: float = 1e-7, out=None,
                  out_dtype=None, plan: Optional[Plan] = None, stream=None):
    """Newton-Schulz steps X = a X + (b X X' + c (X X')^2) X from X = g / (||g|| + eps)
    (gemm_orthogonalize): the orthogonalised update of a weight matrix, or of a
    stack of them.

    g: [m, n] or [batch, m, n], float32, float16 or bfloat16, each matrix row-
    or column-major.  out has g's shape and out_dtype (bfloat16 by default).  A bfloat16
    result is up to 2.2e-3 of its norm from the exact one (3.5e-3 for low ranks); float32 and
    float16 results are within 2e-6 to 4e-5 before their own rounding and take up to three
    times as long.
    Returns `out`."""
    if g.dim() not in (2, 3):
        raise ValueError("g must be [m, n] or [batch, m, n]")
    by_columns = g.stride(-1) != 1 and g.stride(-2) == 1    # then the transposes are row-major
    if out is None:
        out = torch.empty(g.mT.shape if by_columns else g.shape, dtype=out_dtype or torch.bfloat16, device=g.device)
        out = out.mT if by_columns else out
    elif out.shape != g.shape:
        raise ValueError("out must have g's shape")
    device = _device(g, out)
    gv, ov = (g, out) if g.dim() == 3 else (g[None], out[None])
    if by_columns:
        gv, ov = gv.transpose(1, 2), ov.transpose(1, 2)
    batch, m, n = gv.shape
    for t, name in ((gv, "g"), (ov, "out")):
        if (t.stride(2) != 1 and n > 1) or (m > 1 and t.stride(1) < n):
            raise ValueError(f"{name} must have contiguous rows (or columns) like the other")
    ldd = max(ov.stride(1), n, 1)
    stream = _raw_stream(device) if stream is None else stream
    plan = _plan_for(plan, _code(g.dtype), GEMM_F32, device, stream)
    status = _LIB.gemm_orthogonalize(plan.handle, batch, m, n, steps, (ctypes.c_double * 3)(*coeffs), eps,
                                     gv.data_ptr(), max(gv.stride(1), n, 1), gv.stride(0) if batch > 1 else 0,
                                     ov.data_ptr(), ldd, ov.stride(0) if batch > 1 else m * ldd, _code(out.dtype),
                                     stream)
    if status:
        raise GemmError(status, "gemm_orthogonalize")
    return out
