"""Performance cases of the expert-layer operators: products grouped by expert
(forward and backward), products with 4-bit weights (one token to a prompt),
and the orthogonalised update of weight matrices.

`listed()` and `draw()` give cases, `prepare()` a user's data for one of them,
`run()` one pass: in elementary 32-bit torch operations, or, where `own` is
true, through this package's public calls.  `exact()` is the same result in 64
bits and `work()` what a pass cannot do without.
"""
import math

import torch

own = False   # True: run() calls the package's operators

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NS_STEPS = 5
NS_COEFFS = (3.4445, -4.7750, 2.0315)   # the quintic of the Newton-Schulz step
NS_EPS = 1e-7


# ------------------------------- the cases ----------------------------------

def _forward(name, rows, experts, k, n, dtype, bias=False):
    return {"name": name, "op": "forward", "rows": rows, "experts": experts, "k": k, "n": n, "dtype": dtype,
            "bias": bias}


def _backward(name, rows, experts, k, n, dtype):
    return {"name": name, "op": "backward", "rows": rows, "experts": experts, "k": k, "n": n, "dtype": dtype}


def _q4(name, rows, experts, k, n, group, dtype, zeros):
    return {"name": name, "op": "q4", "rows": rows, "experts": experts, "k": k, "n": n, "group": group,
            "dtype": dtype, "zeros": zeros}


def _ortho(name, batch, m, n, dtype):
    return {"name": name, "op": "ortho", "batch": batch, "m": m, "n": n, "dtype": dtype}


def listed():
    return [
        # A decoding step of a small batch: a few tokens, most experts see one or two of them or none.
        _forward("forward_decode", 16, 8, 1024, 2048, "bf16"),
        # A short prompt or a small training batch: ragged, no expert fills a whole tile; bias and ReLU fused.
        _forward("forward_ragged", 1000, 16, 1000, 2048, "f16", bias=True),
        # A training batch over many experts, a few hundred rows each.
        _forward("forward_train", 16384, 64, 2048, 4096, "bf16"),
        # Gradients of a small batch (input and weights).
        _backward("backward_ragged", 777, 8, 512, 1368, "f16"),
        # Gradients of a training batch.
        _backward("backward_train", 16384, 32, 4096, 2048, "bf16"),
        # The update of one small matrix: latency of the chain of products.
        _ortho("ortho_small", 1, 384, 256, "f32"),
        # The updates of a stack of experts' weights, a width that is no multiple of anything.
        _ortho("ortho_experts", 16, 768, 2001, "bf16"),
        # The update of a fully connected layer's weights (4096 x 11008).
        _ortho("ortho_fc", 1, 4096, 11008, "bf16"),
        # One token through a dense layer: the weights are read once.
        _q4("q4_token", 1, 1, 4096, 4096, 128, "f16", False),
        # A few tokens decoded together through a fully connected layer.
        _q4("q4_tokens", 7, 1, 4096, 11008, 64, "bf16", True),
        # A decoding step through experts with 4-bit weights.
        _q4("q4_experts", 24, 16, 2048, 1408, 32, "bf16", False),
        # A prompt through the same layer as the single tokens.
        _q4("q4_prompt", 2000, 1, 4096, 11008, 128, "bf16", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A layer's width: mostly a multiple of 8, as models have them, now and then any number."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.15 else max(lo, v // 8 * 8)


def draw(rng):
    op = rng.choice(["forward", "backward", "ortho", "q4"])
    if op in ("forward", "backward"):
        while True:
            c = {"op": op, "rows": _log(rng, 1, 16384), "experts": _log(rng, 1, 64), "k": _width(rng, 256, 4096),
                 "n": _width(rng, 256, 4096), "dtype": rng.choice(["f16", "bf16"])}
            if c["k"] * c["n"] <= 4096 * 2048:
                break
        if op == "forward":
            c["bias"] = rng.random() < 0.3
        return c
    if op == "ortho":
        while True:
            c = {"op": op, "batch": rng.choice([1, 1, _log(rng, 2, 32)]), "m": _width(rng, 64, 4096),
                 "n": _width(rng, 64, 11008), "dtype": rng.choice(["f32", "bf16"])}
            if _ortho_flops(c) <= 3e12 and c["batch"] * c["m"] * c["n"] <= 2 ** 26:
                return c
    experts = rng.choice([1, 1, _log(rng, 2, 32)])
    while True:
        group = rng.choice([32, 64, 128])
        c = {"op": op, "rows": _log(rng, 1, 2048 if experts == 1 else 256), "experts": experts,
             "k": _log(rng, 512, 11008) // group * group, "n": _log(rng, 512, 11008), "group": group,
             "dtype": rng.choice(["f16", "bf16"]), "zeros": rng.random() < 0.5}
        if experts * c["k"] * c["n"] <= 2 ** 27 and c["rows"] * c["k"] * c["n"] <= 2000 * 4096 * 11008:
            return c


# ------------------------------- the inputs ---------------------------------

def _randn(shape, gen, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _offsets(case, seed):
    """Rows of each expert as a trained router gives them: uneven, some experts without any."""
    gen = torch.Generator().manual_seed(seed)
    if case["experts"] == 1:
        counts = torch.tensor([case["rows"]])
    else:
        p = torch.softmax(0.5 * torch.randn(case["experts"], generator=gen), 0)
        counts = torch.bincount(torch.multinomial(p, case["rows"], True, generator=gen), minlength=case["experts"])
    off = torch.zeros(case["experts"] + 1, dtype=torch.int32)
    off[1:] = counts.cumsum(0)
    return off.cuda(), int(counts.max())


def _quantise(w, group, with_zeros, dtype):
    """Round-to-nearest 4-bit weights with one scale (and zero point) per row and group of K."""
    g = w.unflatten(-1, (-1, group))
    if with_zeros:
        lo, hi = g.amin(-1).clamp(max=0), g.amax(-1).clamp(min=0)
        scale = ((hi - lo) / 15).to(dtype)
        zeros = torch.round(-lo / scale.float()).clamp(0, 15)
    else:
        scale = (g.abs().amax(-1) / 7).to(dtype)
        zeros = torch.full_like(scale, 8, dtype=torch.float32)
    v = (torch.round(g / scale.float()[..., None]) + zeros[..., None]).clamp(0, 15).flatten(-2).to(torch.uint8)
    return v[..., 0::2] | (v[..., 1::2] << 4), scale, zeros.to(torch.uint8) if with_zeros else None


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    st = {"case": case}
    if case["op"] in ("forward", "backward"):
        R, E, K, N = case["rows"], case["experts"], case["k"], case["n"]
        st["offsets"], st["capacity"] = _offsets(case, seed)
        st["x"] = _randn((R, K), gen, 1.0, dt)
        st["w"] = _randn((E, K, N), gen, K ** -0.5, dt)
        if case["op"] == "backward":
            st["dy"] = _randn((R, N), gen, 1.0, dt)
        elif case["bias"]:
            st["bias"] = _randn((E, N), gen, 0.1)
    elif case["op"] == "q4":
        R, E, K, N = case["rows"], case["experts"], case["k"], case["n"]
        st["offsets"], st["capacity"] = _offsets(case, seed)
        st["x"] = _randn((R, K), gen, 1.0, dt)
        parts = [_quantise(_randn((N, K), gen, K ** -0.5), case["group"], case["zeros"], dt) for _ in range(E)]
        st["q"] = torch.stack([p[0] for p in parts])
        st["scales"] = torch.stack([p[1] for p in parts])
        st["zeros"] = torch.stack([p[2] for p in parts]) if case["zeros"] else None
    else:
        # A momentum of gradients: noise with a few strong directions above it.
        B, m, n = case["batch"], case["m"], case["n"]
        r = min(8, m, n)
        strong = 4 * (m ** 0.5 + n ** 0.5) / (m * n) ** 0.5
        g = _randn((B, m, n), gen) + strong * torch.bmm(_randn((B, m, r), gen), _randn((B, r, n), gen))
        st["g"] = (1e-3 * g).to(dt)
    return st


# ------------------------------ the plain forms -----------------------------

def _slots(offsets, rows):
    """The expert of every row and its place among that expert's rows."""
    r = torch.arange(rows, device=offsets.device, dtype=torch.int32)
    e = torch.searchsorted(offsets[1:], r, right=True)
    return e, r.long() - offsets[e]


def _padded(x, e, p, experts, capacity):
    out = torch.zeros((experts, capacity, x.shape[1]), device=x.device)
    out[e, p] = x.float()
    return out


def _weights(st):
    """The values of 4-bit weights: scale * (q - zero)."""
    q = st["q"]
    v = torch.stack((q & 15, q >> 4), -1).flatten(-2).float().unflatten(-1, (-1, st["case"]["group"]))
    z = st["zeros"].float()[..., None] if st["zeros"] is not None else 8.0
    return ((v - z) * st["scales"].float()[..., None]).flatten(-2)


def _plain(st):
    c = st["case"]
    dt = DTYPES[c["dtype"]]
    if c["op"] == "ortho":
        a, b, cc = NS_COEFFS
        x = st["g"].float()
        x = x.transpose(1, 2) if c["m"] > c["n"] else x
        x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
        for _ in range(NS_STEPS):
            s = torch.bmm(x, x.transpose(1, 2))
            x = a * x + torch.bmm(b * s + cc * torch.bmm(s, s), x)
        x = x.transpose(1, 2) if c["m"] > c["n"] else x
        return x.to(torch.bfloat16).contiguous()
    if c["op"] == "q4" and c["experts"] == 1:
        return (st["x"].float() @ _weights(st)[0].t()).to(dt)
    e, p = _slots(st["offsets"], c["rows"])
    x = _padded(st["x"], e, p, c["experts"], st["capacity"])
    if c["op"] == "q4":
        return torch.bmm(x, _weights(st).transpose(1, 2))[e, p].to(dt)
    if c["op"] == "forward":
        y = torch.bmm(x, st["w"].float())
        if c["bias"]:
            y = (y + st["bias"][:, None, :]).clamp(min=0)
        return y[e, p].to(dt)
    dy = _padded(st["dy"], e, p, c["experts"], st["capacity"])
    dx = torch.bmm(dy, st["w"].float().transpose(1, 2))[e, p].to(dt)
    return {"dx": dx, "dw": torch.bmm(x.transpose(1, 2), dy).to(dt)}


# -------------------------- the package's operators -------------------------

_plans = {}


def _plan(G, dtype):
    """A program keeps one plan per operand type."""
    if dtype not in _plans:
        code = {"f32": G.GEMM_F32, "f16": G.GEMM_F16, "bf16": G.GEMM_BF16}[dtype]
        _plans[dtype] = G.Plan(code, G.GEMM_F32, torch.cuda.current_device())
    return _plans[dtype]


def _package(st):
    import dense_gemm_epilogues_gb300 as G
    c = st["case"]
    dt, plan = DTYPES[c["dtype"]], _plan(G, c["dtype"])
    if c["op"] == "forward":
        return G.grouped_matmul(st["x"], st["w"], st["offsets"], bias=st.get("bias"), relu=c["bias"], out_dtype=dt,
                                plan=plan)
    if c["op"] == "backward":
        return {"dx": G.grouped_matmul(st["dy"], st["w"].transpose(1, 2), st["offsets"], out_dtype=dt, plan=plan),
                "dw": G.grouped_weight_grad(st["x"], st["dy"], st["offsets"], out_dtype=dt, plan=plan)}
    if c["op"] == "q4":
        dense = c["experts"] == 1
        return G.q4_matmul(st["x"], st["q"], st["scales"], c["group"], zeros=st["zeros"],
                           offsets=None if dense else st["offsets"], out_dtype=dt, plan=plan)
    return G.orthogonalize(st["g"], steps=NS_STEPS, coeffs=NS_COEFFS, eps=NS_EPS, out_dtype=torch.bfloat16, plan=plan)


def run(state):
    return _package(state) if own else _plain(state)


# ------------------------------ in 64 bits ----------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "ortho":
        a, b, c = NS_COEFFS
        out = []
        for g in st["g"].double():
            y = g / (torch.linalg.vector_norm(g) + NS_EPS)
            for _ in range(NS_STEPS):
                # p(Y) = Y (a + b Y'Y + c (Y'Y)^2), written from whichever side is the shorter one.
                if y.shape[0] <= y.shape[1]:
                    h = y @ y.mT
                    t = h @ y
                    y = a * y + b * t + c * (h @ t)
                else:
                    h = y.mT @ y
                    t = y @ h
                    y = a * y + b * t + c * (t @ h)
            out.append(y)
        return torch.stack(out)
    off = st["offsets"].tolist()
    rows, n = case["rows"], case["n"]
    y = torch.zeros((rows, n), dtype=torch.float64, device="cuda")
    if case["op"] == "q4":
        K, group = case["k"], case["group"]
        k = torch.arange(K, device="cuda")
        for e in range(case["experts"]):
            if off[e] == off[e + 1]:
                continue
            byte = st["q"][e][:, k // 2].double()
            v = torch.where(k % 2 == 1, torch.floor(byte / 16), torch.remainder(byte, 16))
            zero = st["zeros"][e].double()[:, k // group] if case["zeros"] else 8.0
            w = (v - zero) * st["scales"][e].double()[:, k // group]
            y[off[e]:off[e + 1]] = st["x"][off[e]:off[e + 1]].double() @ w.mT
        return y
    dx = torch.zeros((rows, case["k"]), dtype=torch.float64, device="cuda")
    dw = torch.zeros((case["experts"], case["k"], n), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        s = slice(off[e], off[e + 1])
        w, x = st["w"][e].double(), st["x"][s].double()
        if case["op"] == "forward":
            y[s] = x @ w
            if case["bias"]:
                y[s] = torch.relu(y[s] + st["bias"][e].double())
        else:
            dy = st["dy"][s].double()
            dx[s] = dy @ w.mT
            dw[e] = x.mT @ dy
    return y if case["op"] == "forward" else {"dx": dx, "dw": dw}


# ------------------------------- the work -----------------------------------

def _ortho_flops(c):
    """Products of one pass: two symmetric ones (half of their entries) and a full one per step."""
    m, n = min(c["m"], c["n"]), max(c["m"], c["n"])
    return c["batch"] * NS_STEPS * (m * m * n + m * m * m + 2.0 * m * m * n)


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "ortho":
        e = case["batch"] * case["m"] * case["n"]
        return {"bytes": float(e * (size + 2)), "flops": _ortho_flops(case)}
    R, E, K, N = case["rows"], case["experts"], case["k"], case["n"]
    used = E * (1 - (1 - 1 / E) ** R)   # experts that an even router would give a row
    if case["op"] == "q4":
        per = K * N / 2 + K // case["group"] * N * (2 + (1 if case["zeros"] else 0))
        return {"bytes": float(used * per + R * (K + N) * 2), "flops": 2.0 * R * K * N}
    if case["op"] == "forward":
        return {"bytes": float(used * K * N * 2 + R * (K + N) * 2 + (used * N * 4 if case["bias"] else 0)),
                "flops": 2.0 * R * K * N}
    return {"bytes": float(used * K * N * 2 + E * K * N * 2 + R * (2 * K + N) * 2), "flops": 4.0 * R * K * N}
