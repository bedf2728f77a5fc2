"""Plain 64-bit forms of the operators around the products, and the bounds their tests use.

A result rounded once to its type is off by at most U[type] of its value (half a step).  A
sum of n fp32 terms in any order loses at most n 2^-24 of the sum of their absolute values.
expf is within 2 steps (2^-22), and the rounding of its argument x adds |x| 2^-24.
"""
import math

import torch

from expert_helpers import DT, TINY, U  # noqa: F401  (shared with the tests)

EPS = 2.0 ** -23


def within(got, ref, tol, what=""):
    """|got - ref| <= tol, entry by entry; NaN and infinities have to be the same."""
    got, ref = got.double(), ref.double()
    same = (got.isnan() & ref.isnan()) | (got == ref)
    bad = ~(same | ((got - ref).abs() <= tol))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at "
                           f"{bad.nonzero()[0].tolist()}: {got[bad][0]} for {ref[bad][0]}")


def route_ref(logits, top, renormalize=True, mask=None):
    """The routing in 64 bits, choice by choice: (weights, experts, slots, counts, offsets, routed, loss, p, spread)."""
    z = logits.double().cpu()
    T, E = z.shape
    order = torch.where(z.isnan(), math.inf, z)
    nan = z.isnan()
    experts = torch.full((T, top), -1, dtype=torch.long)
    left = order.clone()
    if mask is not None:
        left[~mask.bool().cpu()] = -math.inf
    index = torch.arange(E).expand(T, E)
    for j in range(top):   # NaN before infinity, then by value, then by index
        most = left.amax(1, keepdim=True)
        ties = (left == most) & (most > -math.inf)
        ties = torch.where((ties & nan).any(1, keepdim=True), ties & nan, ties)
        first = torch.where(ties, index, E).amin(1)
        experts[:, j] = torch.where(first < E, first, -1)
        left = torch.where(index == first[:, None], -math.inf, left)
    chosen = experts >= 0
    any_ = chosen[:, :1]
    p = torch.where(any_, torch.softmax(torch.where(any_, z, 0.0), 1), 0.0)
    w = torch.where(chosen, p.gather(1, experts.clamp(min=0)), 0.0)
    if renormalize:
        w = torch.where(chosen, w / w.sum(1, keepdim=True), 0.0)
    counts = torch.bincount(experts[chosen], minlength=E)
    offsets = torch.cat((torch.zeros(1, dtype=torch.long), counts.cumsum(0)))
    flat = torch.where(chosen, experts, E).flatten()
    places = torch.empty_like(flat)
    places[torch.argsort(flat, stable=True)] = torch.arange(flat.numel())
    slots = torch.where(chosen, places.view(T, top), -1)
    rows, routed = int(counts.sum()), int(any_.sum())
    loss = E * (counts * p.sum(0)).sum() / max(1, rows * routed) if rows else torch.tensor(0.0, dtype=torch.float64)
    finite = torch.where(torch.isfinite(z), z, 0.0)
    spread = (finite.amax(1) - finite.amin(1)).max() if T else 0.0
    return w, experts, slots, counts, offsets, routed, loss, p, float(spread)


def route_grad_ref(logits, top, dweights, dloss, renormalize=True, mask=None):
    """(the gradient in 64 bits, the sum of the absolute values of its terms)."""
    w, experts, _, counts, _, routed, _, p, spread = route_ref(logits, top, renormalize, mask)
    T, E = p.shape
    rows = int(counts.sum())
    chosen = experts >= 0
    dw = torch.where(chosen, dweights.double().cpu(), 0.0) if dweights is not None else torch.zeros(T, top, dtype=torch.float64)
    g = (dloss * E * counts / max(1, rows * routed)).expand(T, E).double()
    at = experts.clamp(min=0)
    direct = torch.zeros_like(p)
    mag = torch.zeros_like(p)
    if renormalize:
        direct.scatter_add_(1, at, w * (dw - (w * dw).sum(1, keepdim=True)))
        mag.scatter_add_(1, at, w * (dw.abs() + (w * dw).abs().sum(1, keepdim=True)))
    else:
        g = g.clone().scatter_add_(1, at, dw)
    ga = g.abs()
    any_ = chosen[:, :1]
    ref = torch.where(any_, direct + p * (g - (p * g).sum(1, keepdim=True)), 0.0)
    return ref, mag + p * (ga + (p * ga).sum(1, keepdim=True)), spread


# ------------------------- fully connected layers ---------------------------

ACTS = [None, "relu", "gelu", "gelu_tanh", "silu"]


def act_ref(z, act):
    """(act(z), act'(z)) in 64 bits."""
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act in ("gelu_tanh", "silu"):
        a = 2 * math.sqrt(2 / math.pi)
        u, du = (z, torch.ones_like(z)) if act == "silu" else (a * (z + 0.044715 * z ** 3), a * (1 + 0.134145 * z * z))
        s = torch.sigmoid(u)
        return z * s, s + z * s * torch.sigmoid(-u) * du
    return z, torch.ones_like(z)


def act_error(z, act):
    """How far fp32 activations may be off: the normal distribution by 2.3e-7 (its formula in fp32)
    and two hardware steps (2^-22) of at most 1/2 each, times |z|; a sigmoid by two such steps and
    the rounding of its exponent v, |v| 2^-23 of s(v) with |v| s(v) <= 0.4 where it is not near 1."""
    return 5e-7 * (1 + z.abs()) if act not in (None, "relu") else torch.zeros_like(z)


def act_grad_error(z, act):
    """The same for derivatives: that of the distribution, and of z p(z) the exponential's, two steps
    and z^2 2^-23 with |z|^3 p(z) < 0.5; of sigmoids the product of two, each as above."""
    return 1e-6 * (1 + z.abs()) if act not in (None, "relu") else torch.zeros_like(z)


def linear_ref(x, w, bias, act, residual):
    """(y, z, the error that fp32 sums and the activation may make of y, and of z)."""
    z = x.double() @ w.double()
    mag = x.double().abs() @ w.double().abs()
    if bias is not None:
        z = z + bias.double()
        mag = mag + bias.double().abs()
    ez = (x.shape[1] + 4) * EPS * mag
    y, _ = act_ref(z, act)
    ey = 1.13 * ez + act_error(z, act)   # (no activation is steeper than 1.13)
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2.0 ** -23 * (y.abs() + residual.double().abs())
    return y, z, ey, ez
