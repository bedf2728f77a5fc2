"""Plain 64-bit forms of the expert-layer operators and the error bounds their
tests use.

Bounds (fixed by the arithmetic, not by what a kernel gave): a product is a sum
of K exact or once-rounded terms, added in fp32 in any order with at most
2^-23 of the running magnitude lost by each addition (truncation included), and
rounded once to the output type:
    |D - ref| <= u_out * |ref| + (K + 4) * 2^-23 * (|A| |B|) + the type's smallest step,
with u_out = 2^-8, 2^-11, 2^-24 for bf16, fp16, fp32.
"""
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 1e-38, "f16": 2.0 ** -24, "bf16": 1e-38}


def offsets_of(counts, first=0):
    off = [first]
    for c in counts:
        off.append(off[-1] + c)
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def check(got, ref, mag, depth, out, extra=0.0):
    """got against the 64-bit ref; mag: the same product of absolute values;
    extra: further relative error of each term (rounded operands)."""
    got = got.double()
    tol = U[out] * ref.abs() + ((depth + 4) * 2.0 ** -23 + extra) * (1 + U[out]) * mag + TINY[out]
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outside the bound, first at {bad.nonzero()[0].tolist()}: "
                           f"worst {((got - ref).abs() / tol).nan_to_num(1e9).max():.2f} of it")


def grouped_ref(x, w, offsets, bias=None, relu=False, alpha=1.0):
    """(ref, magnitude); rows of no group are zero."""
    off = offsets.tolist()
    ref = torch.zeros((x.shape[0], w.shape[2]), dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(ref)
    for g in range(w.shape[0]):
        s = slice(off[g], off[g + 1])
        ref[s] = alpha * (x[s].double() @ w[g].double())
        mag[s] = abs(alpha) * (x[s].double().abs() @ w[g].double().abs())
        if bias is not None:
            b = (bias[g] if bias.dim() == 2 else bias).double()
            ref[s] += b
            mag[s] += b.abs()
    return (ref.clamp(min=0) if relu else ref), mag


def wgrad_ref(x, dy, offsets, alpha=1.0, c=None):
    off = offsets.tolist()
    E = len(off) - 1
    ref = torch.zeros((E, x.shape[1], dy.shape[1]), dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(ref)
    for g in range(E):
        s = slice(off[g], off[g + 1])
        ref[g] = alpha * (x[s].double().t() @ dy[s].double())
        mag[g] = abs(alpha) * (x[s].double().abs().t() @ dy[s].double().abs())
    if c is not None:
        ref += c.double()
        mag += c.double().abs()
    return ref, mag


def q4_weights(q, scales, zeros, K, group):
    """w[.., n, k] in 64 bits from the packed form."""
    k = torch.arange(K, device=q.device)
    byte = q.long()[..., k // 2]
    v = torch.where(k % 2 == 1, byte >> 4, byte & 15).double()
    z = zeros.double()[..., k // group] if zeros is not None else 8.0
    return (v - z) * scales.double()[..., k // group]


def newton_schulz_ref(g, steps=5, coeffs=(3.4445, -4.7750, 2.0315), eps=1e-7):
    a, b, c = coeffs
    x = g.double()
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    for _ in range(steps):
        s = x @ x.mT
        x = a * x + (b * s + c * (s @ s)) @ x
    return x


def random_q4(shape_n, K, group, scale_dtype, zeros, gen, groups=None):
    """Random packed weights: every byte, scales in (0, 1), zeros 0..15 or none."""
    lead = () if groups is None else (groups,)
    kg = -(-K // group)
    q = torch.randint(0, 256, lead + (shape_n, (K + 1) // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = (0.1 + torch.rand(lead + (shape_n, kg), device="cuda", generator=gen)).to(scale_dtype)
    z = torch.randint(0, 16, lead + (shape_n, kg), dtype=torch.uint8, device="cuda", generator=gen) if zeros else None
    return q, s, z
