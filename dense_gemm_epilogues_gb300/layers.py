"""What stands around the products of a layer, on torch tensors: fully connected layers with
activation and residual, the routing of tokens to
experts with its balance loss, rows between tokens and experts, gradients clipped by their
global norm.

Like the expert-layer functions these check their arguments, read pointers, strides and the
current stream and call the C entry points of include/gemm.h.  A call without `plan` uses the
default plan of its thread, stream and operand type; nothing is recorded for autograd: each
function's gradient is a function beside it.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

import torch

from . import (GEMM_F32, GEMM_LINEAR_GELU, GEMM_LINEAR_GELU_TANH, GEMM_LINEAR_NONE, GEMM_LINEAR_RELU, GEMM_LINEAR_SILU,
               GEMM_OP_N, GEMM_OP_T, GemmError, Plan, gemm_linear_t, gemm_routing_t, gemm_tensor_t)
from .expert import _LIB, _code, _device, _pitch, _plan_for, _raw_stream

_I32, _F32 = torch.int32, torch.float32
_ACTS = {None: GEMM_LINEAR_NONE, "relu": GEMM_LINEAR_RELU, "gelu": GEMM_LINEAR_GELU,
         "gelu_tanh": GEMM_LINEAR_GELU_TANH, "silu": GEMM_LINEAR_SILU}


def _ld(t, cols: int, name: str) -> int:
    """The pitch of a row-major 2-D tensor."""
    return (cols or 1) if t.is_contiguous() else _pitch(t.shape, t.stride(), name)


# ------------------------- fully connected layers ---------------------------

def _act(name) -> int:
    try:
        return _ACTS[name]
    except KeyError:
        raise ValueError(f"activation {name!r} is not one of {sorted(k for k in _ACTS if k)} or None") from None


def _weights(w, K: int, N: int, name: str = "w"):
    """(layout, leading dimension) of a [K, N] matrix with unit stride along N or K."""
    a, b = w.stride()
    if (b == 1 or N <= 1) and (a >= N or K <= 1):
        return GEMM_OP_T, max(a, N, 1)
    if (a == 1 or K <= 1) and (b >= K or N <= 1):
        return GEMM_OP_N, max(b, K, 1)
    raise ValueError(f"{name} must have unit stride along K or N and no overlapping rows")


def _like(t, shape, dtype, name: str) -> int:
    """The pitch of a row-major tensor that must have this shape and type."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must be {str(dtype)[6:]} of shape {tuple(shape)}")
    return _ld(t, shape[1], name)


def linear(x, w, *, bias=None, activation: Optional[str] = None, residual=None, save_pre: bool = False, out=None,
           out_dtype=None, plan: Optional[Plan] = None, stream=None):
    """A fully connected layer in one kernel (gemm_run_linear):
    z = x @ w + bias;  y = activation(z) + residual.  Returns y, or (y, z) with save_pre: what
    linear_grad needs of an activation.

    x: [rows, K] float16 or bfloat16; w: [K, N] of the same type with unit stride along N or K (a
    transposed [N, K] matrix); bias: [N] of a floating type; residual: [rows, N] of the output's
    type (it may be `out`).  activation: "relu", "gelu", "gelu_tanh", "silu" or None.  out_dtype
    defaults to x's."""
    dtype = x.dtype
    M, K = x.shape
    K2, N = w.shape
    if K2 != K or w.dtype is not dtype:
        raise ValueError("x must be [rows, K] and w [K, N] of the same type")
    act = _act(activation)
    layout, ldb = _weights(w, K, N)
    lda = _ld(x, K, "x")
    device = _device(x, w, bias, residual, out)
    if out is None:
        out_dtype = out_dtype or dtype
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
        ldd = max(N, 1)
    else:
        out_dtype = out.dtype
        ldd = _like(out, (M, N), out_dtype, "out")
    code = _code(out_dtype)
    ldr = _like(residual, (M, N), out_dtype, "residual") if residual is not None else 0
    pre = torch.empty((M, N), dtype=out_dtype, device=x.device) if save_pre else None
    bias_code = GEMM_F32
    if bias is not None:
        if bias.shape != (N,) or (N > 1 and bias.stride(0) != 1):
            raise ValueError("bias must be [N] and contiguous")
        bias_code = _code(bias.dtype)
    stream = _raw_stream(device) if stream is None else stream
    plan = _plan_for(plan, _code(dtype), GEMM_F32, device, stream)
    epi = gemm_linear_t(bias.data_ptr() if bias is not None else None, bias_code, act,
                        residual.data_ptr() if residual is not None else None, ldr,
                        pre.data_ptr() if save_pre else None, max(N, 1), code)
    status = _LIB.gemm_run_linear(plan.handle, layout, M, N, K, x.data_ptr(), lda, w.data_ptr(), ldb, out.data_ptr(),
                                  ldd, epi, stream)
    if status:
        raise GemmError(status, "gemm_run_linear")
    return (out, pre) if save_pre else out


def linear_grad(dy, x, w, *, activation: Optional[str] = None, pre=None, dw_dtype=None, input_grad: bool = True,
                weight_grad: bool = True, bias_grad: bool = True, plan: Optional[Plan] = None, stream=None):
    """(dx, dw, dbias) of linear for its output's gradient dy (gemm_run_linear_grad), None for
    what is not asked for; the residual's gradient is dy itself.

    dy: [rows, N] of x's type; pre: linear's z in x's type, needed with an activation.  dx has x's
    type; dw has w's order of dimensions and dw_dtype (w's type by default); dbias is float32, from
    values that are not rounded."""
    dtype = x.dtype
    M, K = x.shape
    K2, N = w.shape
    if K2 != K or w.dtype is not dtype:
        raise ValueError("x must be [rows, K] and w [K, N] of the same type")
    act = _act(activation)
    layout, ldb = _weights(w, K, N)
    lddy = _like(dy, (M, N), dtype, "dy")
    ldp = 0
    if act != GEMM_LINEAR_NONE:
        if pre is None:
            raise ValueError("an activation's gradient needs pre")
        ldp = _like(pre, (M, N), dtype, "pre")
    device = _device(x, w, dy, pre)
    d = x.device
    dx = torch.empty((M, K), dtype=dtype, device=d) if input_grad else None
    dw_dtype = dw_dtype or dtype
    dw = None
    if weight_grad:
        dw = (torch.empty((K, N), dtype=dw_dtype, device=d) if layout == GEMM_OP_T
              else torch.empty((N, K), dtype=dw_dtype, device=d).t())
    db = torch.empty((N,), dtype=_F32, device=d) if bias_grad else None
    stream = _raw_stream(device) if stream is None else stream
    plan = _plan_for(plan, _code(dtype), GEMM_F32, device, stream)
    status = _LIB.gemm_run_linear_grad(plan.handle, layout, M, N, K, dy.data_ptr(), lddy,
                                       pre.data_ptr() if ldp else None, ldp, act, x.data_ptr(),
                                       _pitch((M, K), x.stride(), "x"), w.data_ptr(), ldb,
                                       dx.data_ptr() if input_grad else None, max(K, 1),
                                       dw.data_ptr() if weight_grad else None,
                                       max(N if layout == GEMM_OP_T else K, 1), _code(dw_dtype),
                                       db.data_ptr() if bias_grad else None, stream)
    if status:
        raise GemmError(status, "gemm_run_linear_grad")
    return dx, dw, db


# ------------------------------- routing ------------------------------------

class Routing(NamedTuple):
    """Tokens routed to experts (route); the gradients and the exchange of rows read it."""
    weights: torch.Tensor    # [tokens, top] float32: what each chosen expert's row is added with
    experts: torch.Tensor    # [tokens, top] int32, best first; -1 behind the last
    slots: torch.Tensor      # [tokens, top] int32: places among the rows sorted by expert; -1
    counts: torch.Tensor     # [experts] int32: rows of each expert
    offsets: torch.Tensor    # [experts + 1] int32, as grouped_matmul takes them
    routed: torch.Tensor     # int32 scalar: tokens that have any expert
    loss: Optional[torch.Tensor] = None   # float32 scalar: the balance loss
    renormalize: bool = True


def _flat(t, dtype, shape, name: str):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {str(dtype)[6:]} tensor of shape {tuple(shape)}")


def _check_routing(r, tokens: int, experts: int):
    shape = r.experts.shape
    if len(shape) != 2 or shape[0] != tokens:
        raise ValueError("the routing is of another number of tokens")
    _flat(r.experts, _I32, shape, "experts")
    _flat(r.slots, _I32, shape, "slots")
    _flat(r.weights, _F32, shape, "weights")
    _flat(r.counts, _I32, (experts,), "counts")
    _flat(r.offsets, _I32, (experts + 1,), "offsets")
    if r.routed.dtype is not _I32 or r.routed.numel() != 1:
        raise ValueError("routed must be an int32 scalar")
    if r.loss is not None and (r.loss.dtype is not _F32 or r.loss.numel() != 1):
        raise ValueError("loss must be a float32 scalar")
    return shape[1]


def _c_routing(r, top: int):
    return gemm_routing_t(r.weights.data_ptr(), r.experts.data_ptr(), r.slots.data_ptr(), r.counts.data_ptr(),
                          r.offsets.data_ptr(), r.routed.data_ptr(), r.loss.data_ptr() if r.loss is not None else None,
                          top, 1 if r.renormalize else 0)


def route(logits, top: int, *, renormalize: bool = True, mask=None, out: Optional[Routing] = None,
          plan: Optional[Plan] = None, stream=None) -> Routing:
    """Routes every token to its `top` largest logits (gemm_route): a Routing with the weights
    (softmax at the chosen experts, adding up to 1 if renormalize), the experts, every row's
    place among the rows sorted by expert, the experts' row counts and offsets, and the balance
    loss  E * sum_e (rows of e / rows) * (mean over tokens of p_e),  1 for an even routing.

    logits: [tokens, experts] float32, float16 or bfloat16 with contiguous rows.  Equal logits
    go to the lower index; an expert at -inf is not taken (its weight is 0, its expert and slot
    -1).  mask: [tokens] bool or uint8, the tokens that count.  out: a Routing to write into."""
    tokens, experts = logits.shape
    if not 0 < top <= experts:
        raise ValueError("top must be between 1 and the number of experts")
    ld = _pitch((tokens, experts), logits.stride(), "logits")
    if mask is not None and (mask.dtype not in (torch.bool, torch.uint8) or mask.shape != (tokens,)
                             or not mask.is_contiguous()):
        raise ValueError("mask must be a contiguous bool or uint8 tensor of one entry per token")
    device = _device(logits, mask)
    if out is None:
        d = logits.device
        r = Routing(torch.empty((tokens, top), dtype=_F32, device=d), torch.empty((tokens, top), dtype=_I32, device=d),
                    torch.empty((tokens, top), dtype=_I32, device=d), torch.empty((experts,), dtype=_I32, device=d),
                    torch.empty((experts + 1,), dtype=_I32, device=d), torch.empty((), dtype=_I32, device=d),
                    torch.empty((), dtype=_F32, device=d), renormalize)
    else:
        if _check_routing(out, tokens, experts) != top:
            raise ValueError("out is of another top")
        _device(logits, out.weights, out.experts, out.slots, out.counts, out.offsets, out.routed, out.loss)
        r = out if out.renormalize == renormalize else out._replace(renormalize=renormalize)
    stream = _raw_stream(device) if stream is None else stream
    plan = _plan_for(plan, _code(logits.dtype), GEMM_F32, device, stream)
    status = _LIB.gemm_route(plan.handle, tokens, experts, logits.data_ptr(), ld,
                             mask.data_ptr() if mask is not None else None, _c_routing(r, top), stream)
    if status:
        raise GemmError(status, "gemm_route")
    return r


def route_grad(logits, routing: Routing, *, dweights=None, dloss=None, out=None, plan: Optional[Plan] = None,
               stream=None):
    """The gradient of a routing's weights and balance loss by its logits (gemm_route_grad), in
    their type and shape; the choice and the counts are constants.

    dweights: [tokens, top] float32, or None.  dloss: a float32 scalar on the device, a number,
    or None (the loss is not used)."""
    tokens, experts = logits.shape
    top = _check_routing(routing, tokens, experts)
    if dweights is not None:
        _flat(dweights, _F32, (tokens, top), "dweights")
    scale, p = 1.0, None
    if dloss is None:
        scale = 0.0
    elif isinstance(dloss, torch.Tensor):
        if dloss.dtype is not _F32 or dloss.numel() != 1:
            raise ValueError("dloss must be a float32 scalar")
        p = dloss.data_ptr()
    else:
        scale = float(dloss)
    if out is None:
        out = torch.empty((tokens, experts), dtype=logits.dtype, device=logits.device)
    elif out.shape != logits.shape or out.dtype is not logits.dtype:
        raise ValueError("out must have the shape and type of logits")
    device = _device(logits, out, dweights, dloss if p is not None else None, routing.weights, routing.experts,
                     routing.counts, routing.offsets, routing.routed)
    stream = _raw_stream(device) if stream is None else stream
    plan = _plan_for(plan, _code(logits.dtype), GEMM_F32, device, stream)
    status = _LIB.gemm_route_grad(plan.handle, tokens, experts, logits.data_ptr(),
                                  _pitch((tokens, experts), logits.stride(), "logits"), _c_routing(routing, top),
                                  dweights.data_ptr() if dweights is not None else None, scale, p, out.data_ptr(),
                                  _pitch((tokens, experts), out.stride(), "out"), stream)
    if status:
        raise GemmError(status, "gemm_route_grad")
    return out


def _slots(routing):
    """The slots of a routing and their shape."""
    slots = routing.slots
    shape = slots.shape
    if slots.dtype is not _I32 or len(shape) != 2 or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous int32 tensor [tokens, top]")
    return slots, shape


def _rows_out(out, rows: int, width: int, like):
    if out is None:
        return torch.empty((rows, width), dtype=like.dtype, device=like.device), width or 1
    if out.shape != (rows, width) or out.dtype is not like.dtype:
        raise ValueError("out must be [rows, width] of the rows' type")
    return out, _ld(out, width, "out")


def _used(routing) -> int:
    """Where the number of rows in use stands: the last offset."""
    e = routing.offsets
    if e.dtype is not _I32 or e.dim() != 1 or not e.is_contiguous() or e.numel() < 1:
        raise ValueError("offsets must be a contiguous int32 tensor")
    return e.data_ptr() + 4 * (e.numel() - 1)


def dispatch(x, routing: Routing, *, out=None, plan: Optional[Plan] = None, stream=None):
    """Every token's row to the places of its experts' rows (gemm_dispatch): [tokens * top, width]
    rows sorted by expert, those behind the last used one zero.  x: [tokens, width] float32,
    float16 or bfloat16 with contiguous rows."""
    slots, (tokens, top) = _slots(routing)
    n, width = x.shape
    if n != tokens:
        raise ValueError("x must have one row per token")
    used, ldx = _used(routing), _ld(x, width, "x")
    rows = tokens * top if out is None else out.shape[0]
    out, ldo = _rows_out(out, rows, width, x)
    device = _device(x, out, slots, routing.offsets)
    stream = _raw_stream(device) if stream is None else stream
    plan = _plan_for(plan, _code(x.dtype), GEMM_F32, device, stream)
    status = _LIB.gemm_dispatch(plan.handle, tokens, top, rows, width, x.data_ptr(), ldx, slots.data_ptr(), used,
                                out.data_ptr(), ldo, stream)
    if status:
        raise GemmError(status, "gemm_dispatch")
    return out


def _combine(y, routing, weights, residual, out, plan, stream):
    slots, shape = _slots(routing)
    tokens, top = shape
    rows, width = y.shape
    w = r = None
    ldr = 0
    if weights is not None:
        _flat(weights, _F32, shape, "weights")
        w = weights.data_ptr()
    if residual is not None:
        if residual.shape != (tokens, width) or residual.dtype is not y.dtype:
            raise ValueError("residual must be [tokens, width] of y's type")
        r, ldr = residual.data_ptr(), _ld(residual, width, "residual")
    ldy = _ld(y, width, "y")
    out, ldo = _rows_out(out, tokens, width, y)
    device = _device(y, out, slots, weights, residual)
    stream = _raw_stream(device) if stream is None else stream
    plan = _plan_for(plan, _code(y.dtype), GEMM_F32, device, stream)
    status = _LIB.gemm_combine(plan.handle, tokens, top, rows, width, y.data_ptr(), ldy, slots.data_ptr(), w, r, ldr,
                               out.data_ptr(), ldo, stream)
    if status:
        raise GemmError(status, "gemm_combine")
    return out


def combine(y, routing: Routing, *, residual=None, out=None, plan: Optional[Plan] = None, stream=None):
    """The experts' rows back to their tokens (gemm_combine):
    out[t] = residual[t] + sum_j weights[t, j] * y[slots[t, j]], [tokens, width] of y's type.

    y: [rows, width] sorted rows; residual: [tokens, width] of y's type (it may be `out`).  Sums
    are fp32; for a result or a residual of fp32 beside 16-bit experts y goes in as fp32 (y.float(),
    or the product's out_dtype)."""
    return _combine(y, routing, routing.weights, residual, out, plan, stream)


def dispatch_grad(drows, routing: Routing, *, out=None, plan: Optional[Plan] = None, stream=None):
    """The gradient of dispatch: the sum of every token's rows of drows (gemm_combine with
    weights of one)."""
    return _combine(drows, routing, None, None, out, plan, stream)


def combine_grad(dout, y, routing: Routing, *, out=None, plan: Optional[Plan] = None, stream=None):
    """(dy, dweights) of combine (gemm_combine_grad): dy like y, rows behind the last used one
    zero; dweights [tokens, top] float32, 0 where there is no row.  The residual's gradient is
    dout itself.  out: where dy goes."""
    slots, shape = _slots(routing)
    tokens, top = shape
    rows, width = y.shape
    if dout.shape != (tokens, width) or dout.dtype is not y.dtype:
        raise ValueError("dout must be [tokens, width] of y's type")
    weights = routing.weights
    _flat(weights, _F32, shape, "weights")
    used, ldd, ldy = _used(routing), _ld(dout, width, "dout"), _ld(y, width, "y")
    out, ldo = _rows_out(out, rows, width, y)
    device = _device(y, out, slots, dout, weights, routing.offsets)
    dweights = torch.empty(shape, dtype=_F32, device=y.device)
    stream = _raw_stream(device) if stream is None else stream
    plan = _plan_for(plan, _code(y.dtype), GEMM_F32, device, stream)
    status = _LIB.gemm_combine_grad(plan.handle, tokens, top, rows, width, dout.data_ptr(), ldd, y.data_ptr(), ldy,
                                    slots.data_ptr(), used, weights.data_ptr(), out.data_ptr(), ldo,
                                    dweights.data_ptr(), stream)
    if status:
        raise GemmError(status, "gemm_combine_grad")
    return out, dweights


# ------------------------------ clipping ------------------------------------

def _fills(t) -> bool:
    """Do the tensor's entries fill a stretch of memory, in any order of its dimensions?"""
    if t.is_contiguous():
        return True
    need = 1
    for stride, size in sorted(zip(t.stride(), t.shape)):
        if size == 1:
            continue
        if stride != need:
            return False
        need *= size
    return True


class TensorList:
    """Tensors whose global norm is taken and that are scaled together, laid out once: the
    gradients that a program keeps from step to step (a tensor that has other memory by the time
    of a call is refused).  out: where the scaled values go, tensors of the same shapes and
    strides and any of the types, or None for one that only counts (out=None: all in place).
    What is written may not share memory with any other entry."""

    def __init__(self, tensors, out=None):
        self.tensors, self.out = list(tensors), list(out) if out is not None else None
        to = self.tensors if self.out is None else self.out
        if len(to) != len(self.tensors):
            raise ValueError("out must have a tensor for each")
        self.table = (gemm_tensor_t * max(1, len(to)))()
        spans = []
        for i, (t, o) in enumerate(zip(self.tensors, to)):
            if not _fills(t):
                raise ValueError("tensors must fill their memory (no gaps between their entries)")
            if o is not None and o is not t and (o.shape != t.shape or o.stride() != t.stride()):
                raise ValueError("out must have the tensors' shapes and strides")
            n, code = t.numel(), _code(t.dtype)
            self.table[i] = gemm_tensor_t(t.data_ptr(), o.data_ptr() if o is not None else None, n, code,
                                          _code(o.dtype) if o is not None else code)
            if n:
                spans.append((t.data_ptr(), t.data_ptr() + n * t.element_size(), i, o is t))
                if o is not None and o is not t:
                    spans.append((o.data_ptr(), o.data_ptr() + n * o.element_size(), i, True))
        spans.sort()
        end, written_end = 0, 0   # of all spans so far, and of those that are written
        for lo, hi, i, written in spans:
            if lo < (end if written else written_end):
                raise ValueError("tensors overlap")
            end = max(end, hi)
            written_end = max(written_end, hi) if written else written_end
        self.device = _device(*self.tensors, *(self.out or ())) if self.tensors else None
        self._all = self.tensors + [o for o in self.out or () if o is not None]
        self._at = list(map(torch.Tensor.data_ptr, self._all))
        self._read = None

    def read_table(self):
        """The table without places to write to, laid out once too."""
        if self._read is None:
            self._read = type(self.table)(*(gemm_tensor_t(e.src, None, e.count, e.src_type, e.src_type) for e in self.table))
        return self._read

    def check(self):
        if list(map(torch.Tensor.data_ptr, self._all)) != self._at:
            raise ValueError("a tensor of the list has moved")


def _norm_of(tensors, max_norm: float, eps: float, scales: bool, plan, stream):
    if isinstance(tensors, TensorList):
        tensors.check()
    else:
        tensors = list(tensors)
        tensors = TensorList(tensors, None if scales else [None] * len(tensors))
    if not max_norm >= 0 or not 0 <= eps < math.inf:
        raise ValueError("max_norm and eps must not be negative, and eps finite")
    device = tensors.device
    if device is None:
        device = plan.device if plan is not None else torch.cuda.current_device()
        norm = torch.empty((), dtype=_F32, device=f"cuda:{device}")
    else:
        norm = torch.empty((), dtype=_F32, device=tensors.tensors[0].device)
    stream = _raw_stream(device) if stream is None else stream
    if plan is None:
        plan = _plan_for(None, GEMM_F32, GEMM_F32, device, stream)
    elif plan.device != device:
        raise ValueError("the plan is on another device")
    table = tensors.table if scales else tensors.read_table()
    status = _LIB.gemm_clip_norm(plan.handle, len(tensors.tensors), table, max_norm, eps, norm.data_ptr(), stream)
    if status:
        raise GemmError(status, "gemm_clip_norm")
    return norm


def clip_grad_norm(tensors, max_norm: float, *, eps: float = 1e-6, plan: Optional[Plan] = None, stream=None):
    """Scales tensors by min(1, max_norm / (norm + eps)) of their global norm (gemm_clip_norm) and
    returns the norm, a float32 scalar on the device.  A norm that is not finite leaves the
    values as they are, so that the step can be skipped.

    tensors: a list of float32, float16 and bfloat16 tensors (scaled in place) or a TensorList,
    which may send the scaled values elsewhere and in another type.  None may overlap another.
    The plan may be of any type."""
    return _norm_of(tensors, max_norm, eps, True, plan, stream)


def grad_norm(tensors, *, plan: Optional[Plan] = None, stream=None):
    """The global norm of a list of tensors or a TensorList, a float32 scalar on the device.  The
    tensors are only read: a list may name the same memory twice, and counts it as often."""
    return _norm_of(tensors, math.inf, 0.0, False, plan, stream)
