"""Performance cases of the operators around the products: fully connected layers with
bias, activation and residual (forward and backward), routing of tokens to experts with
its balance loss (and gradient), the exchange of rows between tokens and experts (both
directions), and gradients clipped by their global norm.

`listed()` and `draw()` give cases, `prepare()` a user's data for one of them,
`run()` one pass: in elementary 32-bit torch operations, or, where `own` is
true, through this package's public calls.  `exact()` is the same result in 64
bits and `work()` what a pass cannot do without.
"""
import itertools
import math

import torch

own = False   # True: run() calls the package's operators

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CLIP_EPS = 1e-6


# ------------------------------- the cases ----------------------------------

def _linear(name, rows, k, n, dtype, act, bias=False, residual=False, save=False, layout="kn"):
    return {"name": name, "op": "linear", "rows": rows, "k": k, "n": n, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "save": save, "layout": layout}


def _linear_grad(name, rows, k, n, dtype, act, layout="kn"):
    return {"name": name, "op": "linear_grad", "rows": rows, "k": k, "n": n, "dtype": dtype, "act": act,
            "layout": layout}


def _route(name, op, tokens, experts, top, dtype, renormalize=True, padded=False):
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "top": top, "dtype": dtype,
            "renormalize": renormalize, "padded": padded}


def _exchange(name, op, tokens, top, d, dtype, experts, padded=False):
    return {"name": name, "op": op, "tokens": tokens, "top": top, "d": d, "dtype": dtype, "experts": experts,
            "padded": padded}


def _clip(name, layers, k, n, experts, odd, dtype, out):
    return {"name": name, "op": "clip", "layers": layers, "k": k, "n": n, "experts": experts, "odd": odd,
            "dtype": dtype, "out": out}


def listed():
    return [
        # One token through a fully connected layer: the weights are read once.
        _linear("linear_token", 1, 4096, 11008, "bf16", "silu"),
        # A short prompt, no size a whole number of tiles: bias, activation and residual fused.
        _linear("linear_ragged", 1000, 1000, 2048, "f16", "gelu_tanh", bias=True, residual=True),
        # The fully connected layer of a training step, which keeps what the activation was applied to.
        _linear("linear_train", 8192, 4096, 11008, "bf16", "gelu", bias=True, save=True),
        # Its gradients: of the input, the weights and the bias.
        _linear_grad("linear_backward", 4096, 4096, 11008, "bf16", "gelu"),
        # The router of a decoding step of a small batch.
        _route("route_decode", "route", 16, 8, 2, "f32"),
        # The router of a padded training batch.
        _route("route_train", "route", 16384, 64, 6, "f32", padded=True),
        # Its gradient: of the weights that the experts' outputs are added with, and of the balance loss.
        _route("route_backward", "route_grad", 16384, 64, 6, "bf16", padded=True),
        # Rows to and from the experts in a decoding step.
        _exchange("exchange_decode", "exchange", 16, 2, 1024, "bf16", 8),
        # The same for a padded training batch.
        _exchange("exchange_train", "exchange", 16384, 2, 2048, "bf16", 64, padded=True),
        # Its gradients: of the experts' outputs, of the weights and of the tokens.
        _exchange("exchange_backward", "exchange_grad", 8191, 4, 4096, "f16", 32),
        # The gradients of a small expert layer.
        _clip("clip_small", 1, 256, 512, 8, 3, "f32", "f32"),
        # The fp32 gradients of a few layers with experts and many small vectors, handed on in bf16.
        _clip("clip_layers", 4, 2048, 1408, 16, 150, "f32", "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A layer's width: mostly a multiple of 8, as models have them, now and then any number."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.15 else max(lo, v // 8 * 8)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "route", "route_grad", "exchange", "exchange_grad", "clip"])
    dtype = rng.choice(["f16", "bf16"])
    if op in ("linear", "linear_grad"):
        while True:
            c = {"op": op, "rows": _log(rng, 1, 8192), "k": _width(rng, 256, 11008), "n": _width(rng, 256, 11008),
                 "dtype": dtype, "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                 "layout": rng.choice(["kn", "nk"])}
            if c["rows"] * c["k"] * c["n"] <= 4096 * 4096 * 11008:
                break
        if op == "linear":
            c.update(bias=rng.random() < 0.5, residual=rng.random() < 0.5, save=rng.random() < 0.3)
        return c
    if op in ("route", "route_grad"):
        experts = _log(rng, 4, 512)
        while True:
            c = {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts, "top": min(experts, _log(rng, 1, 8)),
                 "dtype": rng.choice(["f32", "f16", "bf16"]), "renormalize": rng.random() < 0.7,
                 "padded": rng.random() < 0.5}
            if c["tokens"] * experts <= 2 ** 20:
                return c
    if op in ("exchange", "exchange_grad"):
        while True:
            c = {"op": op, "tokens": _log(rng, 1, 16384), "top": _log(rng, 1, 8), "d": _width(rng, 256, 8192),
                 "dtype": dtype, "padded": rng.random() < 0.5}
            c["experts"] = max(c["top"], _log(rng, 4, 128))
            if c["tokens"] * c["top"] * c["d"] <= 2 ** 26:
                return c
    while True:
        c = {"op": op, "layers": _log(rng, 1, 16), "k": _width(rng, 128, 4096), "n": _width(rng, 128, 4096),
             "experts": _log(rng, 1, 32), "odd": _log(rng, 1, 300), "dtype": rng.choice(["f32", "bf16"])}
        c["out"] = rng.choice([c["dtype"], "bf16"])
        if c["layers"] * c["k"] * c["n"] * c["experts"] <= 4 * 2048 * 1408 * 16:
            return c


# ------------------------------- the inputs ---------------------------------

def _randn(shape, gen, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _logits(tokens, experts, gen):
    """A trained router's logits: some experts are liked more than others."""
    return _randn((tokens, experts), gen) + _randn((1, experts), gen, 0.5)


def _mask(tokens):
    """Which tokens of a padded batch count: of four sequences, each a part."""
    t = torch.arange(tokens, device="cuda")
    length = max(1, -(-tokens // 4))
    return t % length < length - (t // length) * length // 8


def _top(logits, top, mask, experts):
    """(experts [T, k], logits [T, k]) in falling order of the logits, the lowest index first where
    they are equal; an expert whose logit is -inf, and any of a token that does not count, is -1."""
    value, index = torch.sort(logits, dim=1, descending=True, stable=True)
    value, index = value[:, :top], index[:, :top]
    used = value != -math.inf
    if mask is not None:
        used = used & mask[:, None]
    return torch.where(used, index, -1).int(), value


def _rows(index, experts):
    """(slots, counts, offsets, routed): the place of every (token, expert) among the rows sorted by expert, the
    rows of every expert, where they begin, and how many tokens have any."""
    flat = torch.where(index < 0, experts, index).flatten().long()
    place = torch.argsort(torch.argsort(flat, stable=True), stable=True)
    counts = (flat[:, None] == torch.arange(experts, device=flat.device)).sum(0).int()
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0).int()))
    routed = (index[:, 0] >= 0).sum().int()
    return torch.where(index < 0, -1, place.view(index.shape)).int(), counts, offsets, routed


def _shapes(case):
    """The gradients of `layers` expert layers (two stacks of matrices, a bias) and `odd` vectors."""
    k, n, e = case["k"], case["n"], case["experts"]
    shapes = [(e, k, n), (e, n), (e, n, k)] * case["layers"]
    return shapes + [(1 + (i * 977) % (2 * k),) for i in range(case["odd"])]


def _buffer(case, dt):
    """One buffer for all clipped gradients, as an update that takes them keeps it: (the buffer, a view for
    each, from a multiple of 64 entries on)."""
    shapes = _shapes(case)
    starts = [0]
    starts.extend(itertools.accumulate(-(-math.prod(s) // 64) * 64 for s in shapes))
    flat = torch.zeros(starts[-1], dtype=dt, device="cuda")
    return flat, [flat[a:a + math.prod(s)].view(s) for a, s in zip(starts, shapes)]


def _weight(case, gen, dt):
    k, n = case["k"], case["n"]
    if case["layout"] == "kn":
        return _randn((k, n), gen, k ** -0.5, dt)
    return _randn((n, k), gen, k ** -0.5, dt).t()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op, st = case["op"], {"case": case}
    if op in ("linear", "linear_grad"):
        R, K, N = case["rows"], case["k"], case["n"]
        st["x"], st["w"] = _randn((R, K), gen, 1.0, dt), _weight(case, gen, dt)
        if op == "linear_grad":
            st["pre"] = _randn((R, N), gen, 1.0, dt)
            st["dy"] = _randn((R, N), gen, 1.0, dt)
        else:
            st["bias"] = _randn((N,), gen, 0.1) if case["bias"] else None
            st["residual"] = _randn((R, N), gen, 1.0, dt) if case["residual"] else None
    elif op in ("route", "route_grad"):
        T, E, k = case["tokens"], case["experts"], case["top"]
        st["logits"] = _logits(T, E, gen).to(dt)
        st["mask"] = _mask(T) if case["padded"] else None
        if op == "route_grad":   # what the forward pass left
            st["experts"], _ = _top(st["logits"].float(), k, st["mask"], E)
            st["slots"], st["counts"], st["offsets"], st["routed"] = _rows(st["experts"], E)
            z = st["logits"].double()
            s = torch.where(st["experts"] < 0, 0.0, z.softmax(1).gather(1, st["experts"].long().clamp(min=0)))
            if case["renormalize"]:
                s = s / s.sum(1, keepdim=True).clamp(min=1e-300)
            st["weights"] = s.float()
            st["dweights"] = _randn((T, k), gen)
            st["dloss"] = torch.full((), 0.01 * T, device="cuda")
        st["keep"] = T <= 64   # a decoding loop keeps the buffers of its router
    elif op in ("exchange", "exchange_grad"):
        T, k, d, E = case["tokens"], case["top"], case["d"], case["experts"]
        st["experts"], value = _top(_logits(T, E, gen), k, _mask(T) if case["padded"] else None, E)
        st["slots"], st["counts"], st["offsets"], st["routed"] = _rows(st["experts"], E)
        st["weights"] = torch.where(st["experts"] < 0, 0.0, value.softmax(1))
        st["y"] = _randn((T * k, d), gen, 1.0, dt)
        if op == "exchange":
            st["x"] = _randn((T, d), gen, 1.0, dt)
        else:
            st["dout"] = _randn((T, d), gen, 1.0, dt)
            st["drows"] = _randn((T * k, d), gen, 1.0, dt)
    else:
        # Gradients of some layers are larger than those of others.
        st["g"] = [_randn(s, gen, 1e-3 * (1 + i % 5), dt) for i, s in enumerate(_shapes(case))]
        st["flat"], st["out"] = _buffer(case, DTYPES[case["out"]])
    return st


# ------------------------------ the plain forms -----------------------------

def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _probabilities(z, used):
    """Softmax of the rows of z; zero in a row that counts nowhere."""
    e = torch.exp(z - torch.where(used, z.amax(1, keepdim=True), 0.0))
    return torch.where(used, e / e.sum(1, keepdim=True), 0.0)


def _balance(counts, experts):
    """What an expert's probability adds to the balance loss: its share of the rows, times experts."""
    return experts * counts.float() / counts.sum().clamp(min=1)


def _token_rows(st):
    """(used, rows, tokens): the pairs of a token and a row, flat."""
    k = st["case"]["top"]
    slots = st["slots"].flatten().long()
    used = slots >= 0
    return used, slots.clamp(min=0), torch.arange(slots.numel(), device=slots.device) // k


def _plain(st):
    c = st["case"]
    dt = DTYPES[c["dtype"]]
    op = c["op"]
    if op == "linear":
        z = st["x"].float() @ st["w"].float()
        if c["bias"]:
            z = z + st["bias"]
        y = _act(z, c["act"])
        if c["residual"]:
            y = y + st["residual"].float()
        return {"y": y.to(dt), "pre": z.to(dt)} if c["save"] else y.to(dt)
    if op == "linear_grad":
        dz = st["dy"].float() * _act_grad(st["pre"].float(), c["act"])
        dw = st["x"].float().t() @ dz
        return {"dx": (dz @ st["w"].float().t()).to(dt), "dw": dw.to(dt), "db": dz.sum(0)}
    if op == "route":
        E, k = c["experts"], c["top"]
        z = st["logits"].float()
        index, value = _top(z, k, st["mask"], E)
        slots, counts, offsets, routed = _rows(index, E)
        used = index[:, :1] >= 0
        p = _probabilities(z, used)
        w = torch.where(index >= 0, p.gather(1, index.long().clamp(min=0)), 0.0)
        if c["renormalize"]:
            e = torch.where(index >= 0, torch.exp(value - torch.where(used, value[:, :1], 0.0)), 0.0)
            w = torch.where(used, e / e.sum(1, keepdim=True), 0.0)
        loss = (_balance(counts, E) * p.sum(0)).sum() / routed.clamp(min=1)
        return {"weights": w, "experts": index, "slots": slots, "counts": counts, "offsets": offsets,
                "routed": routed, "loss": loss}
    if op == "route_grad":
        E = c["experts"]
        used = st["experts"][:, :1] >= 0
        p = _probabilities(st["logits"].float(), used)
        g = (st["dloss"] / st["routed"].clamp(min=1)) * _balance(st["counts"], E).expand_as(p)
        chosen = st["experts"] >= 0
        dw = torch.where(chosen, st["dweights"], 0.0)
        at = st["experts"].long().clamp(min=0)
        if c["renormalize"]:
            w = st["weights"]
            direct = torch.zeros_like(p).scatter_add_(1, at, w * (dw - (w * dw).sum(1, keepdim=True)))
        else:
            g = g.scatter_add(1, at, dw)
            direct = 0.0
        return (direct + p * (g - (p * g).sum(1, keepdim=True))).to(dt)
    if op == "exchange":
        used, rows, tokens = _token_rows(st)
        sent = torch.zeros_like(st["y"])
        sent[rows[used]] = st["x"][tokens[used]]
        y = torch.where(used[:, None], st["y"].float()[rows], 0.0) * st["weights"].flatten()[:, None]
        out = st["x"].float() + y.view(c["tokens"], c["top"], c["d"]).sum(1)
        return {"rows": sent, "out": out.to(dt)}
    if op == "exchange_grad":
        used, rows, tokens = _token_rows(st)
        dout = st["dout"].float()[tokens]
        dy = torch.zeros_like(st["y"])
        dy[rows[used]] = (st["weights"].flatten()[:, None] * dout)[used].to(dt)
        dw = torch.where(used, (dout * st["y"].float()[rows]).sum(1), 0.0).view(c["tokens"], c["top"])
        dx = torch.where(used[:, None], st["drows"].float()[rows], 0.0).view(c["tokens"], c["top"], c["d"]).sum(1)
        return {"dy": dy, "dweights": dw, "dx": dx.to(dt)}
    norm = torch.stack([g.float().square().sum() for g in st["g"]]).double().sum().sqrt().float()
    scale = torch.where(torch.isfinite(norm), (1.0 / (norm + CLIP_EPS)).clamp(max=1.0), 1.0)
    _ = [o.copy_(g.float() * scale) for g, o in zip(st["g"], st["out"])]
    return {"norm": norm, "g": st["flat"]}


# -------------------------- the package's operators -------------------------

_plans = {}


def _plan(G, dtype):
    """A program keeps one plan per operand type."""
    if dtype not in _plans:
        code = {"f32": G.GEMM_F32, "f16": G.GEMM_F16, "bf16": G.GEMM_BF16}[dtype]
        _plans[dtype] = G.Plan(code, G.GEMM_F32, torch.cuda.current_device())
    return _plans[dtype]


def _routing(G, st):
    c = st["case"]
    return G.Routing(st["weights"], st["experts"], st["slots"], st["counts"], st["offsets"], st["routed"],
                     renormalize=c.get("renormalize", True))


def _package(st):
    import dense_gemm_epilogues_gb300 as G
    c = st["case"]
    op, plan = c["op"], _plan(G, c["dtype"])
    if op == "linear":
        act = None if c["act"] == "none" else c["act"]
        r = G.linear(st["x"], st["w"], bias=st["bias"], activation=act, residual=st["residual"],
                     save_pre=c["save"], plan=plan)
        return {"y": r[0], "pre": r[1]} if c["save"] else r
    if op == "linear_grad":
        act = None if c["act"] == "none" else c["act"]
        dx, dw, db = G.linear_grad(st["dy"], st["x"], st["w"], activation=act, pre=st["pre"], plan=plan)
        return {"dx": dx, "dw": dw, "db": db}
    if op == "route":
        r = G.route(st["logits"], c["top"], renormalize=c["renormalize"], mask=st["mask"], out=st.get("out"), plan=plan)
        if st["keep"]:
            st["out"] = r
        return {"weights": r.weights, "experts": r.experts, "slots": r.slots, "counts": r.counts,
                "offsets": r.offsets, "routed": r.routed, "loss": r.loss}
    if op == "route_grad":
        return G.route_grad(st["logits"], _routing(G, st), dweights=st["dweights"], dloss=st["dloss"], plan=plan)
    if op == "exchange":
        r = _routing(G, st)
        return {"rows": G.dispatch(st["x"], r, plan=plan), "out": G.combine(st["y"], r, residual=st["x"], plan=plan)}
    if op == "exchange_grad":
        r = _routing(G, st)
        dy, dw = G.combine_grad(st["dout"], st["y"], r, plan=plan)
        return {"dy": dy, "dweights": dw, "dx": G.dispatch_grad(st["drows"], r, plan=plan)}
    if "list" not in st:   # a program's gradients and their places stay from step to step
        st["list"] = G.TensorList(st["g"], out=st["out"])
    norm = G.clip_grad_norm(st["list"], 1.0, eps=CLIP_EPS)
    return {"norm": norm, "g": st["flat"]}


def run(state):
    return _package(state) if own else _plain(state)


# ------------------------------ in 64 bits ----------------------------------

def _exact_act(z, act):
    """(act(z), act'(z))"""
    one = torch.ones_like(z)
    if act == "relu":
        return torch.relu(z), torch.heaviside(z, torch.zeros_like(z))
    if act == "gelu":
        phi = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act in ("gelu_tanh", "silu"):   # z s(u), with u = z or 2 sqrt(2 / pi) (z + 0.044715 z^3)
        a = 2 * math.sqrt(2 / math.pi)
        u, du = (z, one) if act == "silu" else (a * (z + 0.044715 * z ** 3), a * (1 + 0.134145 * z ** 2))
        s = torch.sigmoid(u)
        return z * s, s + z * s * torch.sigmoid(-u) * du
    return z, one


def _exact_route(case, logits, mask):
    """(experts, weights, p) token by token from the definition, all tokens at once: the top experts
    are taken one after the other."""
    z = logits.double()
    T, E = z.shape
    left = z.clone()
    if mask is not None:
        left[~mask] = -math.inf
    index = torch.full((T, case["top"]), -1, dtype=torch.long, device=z.device)
    e = torch.arange(E, device=z.device).expand(T, E)
    for j in range(case["top"]):
        best = left.max(1).values
        first = torch.where((left == best[:, None]) & (left > -math.inf), e, E).min(1).values
        index[:, j] = torch.where(first < E, first, -1)
        left = torch.where(e == first[:, None], -math.inf, left)
    chosen = index >= 0
    p = torch.where(chosen[:, :1], torch.softmax(z, 1).nan_to_num(0.0), 0.0)
    w = torch.where(chosen, p.gather(1, index.clamp(min=0)), 0.0)
    if case["renormalize"]:
        w = torch.where(chosen, w / w.sum(1, keepdim=True), 0.0)
    return index, w, p


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        z = st["x"].double() @ st["w"].double()
        if st["bias"] is not None:
            z += st["bias"].double()
        y = _exact_act(z, case["act"])[0]
        if st["residual"] is not None:
            y = y + st["residual"].double()
        return {"y": y, "pre": z} if case["save"] else y
    if op == "linear_grad":
        dz = st["dy"].double() * _exact_act(st["pre"].double(), case["act"])[1]
        return {"dx": dz @ st["w"].double().mT, "dw": st["x"].double().mT @ dz, "db": dz.sum(0)}
    if op in ("route", "route_grad"):
        E = case["experts"]
        index, w, p = _exact_route(case, st["logits"], st["mask"])
        counts = torch.bincount(index[index >= 0], minlength=E).double()
        tokens, rows = (index[:, 0] >= 0).sum().clamp(min=1), counts.sum().clamp(min=1)
        if op == "route":
            return {"weights": w, "experts": None, "slots": None, "counts": None, "offsets": None,
                    "routed": None, "loss": E / (rows * tokens) * (counts * p.sum(0)).sum()}
        out = torch.zeros_like(p)
        dw = st["dweights"].double()
        for j in range(case["top"]):   # each chosen weight's Jacobian in turn
            at = index[:, j].clamp(min=0)[:, None]
            hit = (index[:, j] >= 0)[:, None]
            gain = torch.where(hit, w[:, j:j + 1] * dw[:, j:j + 1], 0.0)
            if case["renormalize"]:   # d w_j / d z_i = w_j ([i = j] - w_i), i among the chosen ones
                wide = torch.zeros_like(p)
                for i in range(case["top"]):
                    wide.scatter_add_(1, index[:, i].clamp(min=0)[:, None],
                                      torch.where(index[:, i:i + 1] >= 0, w[:, i:i + 1], 0.0))
                out -= gain * wide
            else:                     # d p_j / d z_i = p_j ([i = j] - p_i)
                out -= gain * p
            out.scatter_add_(1, at, gain)
        share = E * counts / (rows * tokens)
        out += float(st["dloss"]) * p * (share - (p @ share)[:, None])
        return out
    if op in ("exchange", "exchange_grad"):
        T, k, d = case["tokens"], case["top"], case["d"]
        w = st["weights"].double()
        if op == "exchange":
            rows, out = torch.zeros((T * k, d), dtype=torch.float64, device="cuda"), st["x"].double()
        else:
            rows, out = torch.zeros((T * k, d), dtype=torch.float64, device="cuda"), torch.zeros_like(st["dout"]).double()
            dw = torch.zeros_like(w)
        for j in range(k):
            t = torch.nonzero(st["slots"][:, j] >= 0)[:, 0]
            r = st["slots"][t, j].long()
            if op == "exchange":
                rows[r] = st["x"][t].double()
                out[t] += w[t, j, None] * st["y"][r].double()
            else:
                rows[r] = w[t, j, None] * st["dout"][t].double()
                dw[t, j] = torch.einsum("td,td->t", st["dout"][t].double(), st["y"][r].double())
                out[t] += st["drows"][r].double()
        return {"rows": rows, "out": out} if op == "exchange" else {"dy": rows, "dweights": dw, "dx": out}
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in st["g"]))
    scale = min(1.0, 1.0 / (norm + CLIP_EPS))
    flat, views = _buffer(case, torch.float64)
    for v, g in zip(views, st["g"]):
        v.copy_(g.double() * scale)
    return {"norm": torch.tensor(norm, dtype=torch.float64), "g": flat}


# ------------------------------- the work -----------------------------------

def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "f32" else 2
    if op in ("linear", "linear_grad"):
        R, K, N = case["rows"], case["k"], case["n"]
        if op == "linear":
            wide = R * N * (1 + case["residual"] + case["save"])
            return {"bytes": float((K * N + R * K + wide) * size + (4 * N if case["bias"] else 0)), "flops": 2.0 * R * K * N}
        return {"bytes": float((2 * K * N + 2 * R * K + 2 * R * N) * size + 4 * N), "flops": 4.0 * R * K * N}
    if op in ("route", "route_grad"):
        T, E, k = case["tokens"], case["experts"], case["top"]
        if op == "route":
            return {"bytes": float(T * E * size + T * k * 12 + 8 * E + (T if case["padded"] else 0)), "flops": 8.0 * T * E}
        return {"bytes": float(2 * T * E * size + T * k * 12 + 4 * E), "flops": 10.0 * T * E}
    if op in ("exchange", "exchange_grad"):
        T, k, d = case["tokens"], case["top"], case["d"]
        if op == "exchange":   # x is read once, by the exchange or as the residual
            return {"bytes": float((2 * T * k * d + 2 * T * d) * size + T * k * 8), "flops": 2.0 * T * k * d}
        return {"bytes": float((3 * T * k * d + 2 * T * d) * size + T * k * 12), "flops": 4.0 * T * k * d}
    n = sum(math.prod(s) for s in _shapes(case))
    return {"bytes": float(n * (size + (4 if case["out"] == "f32" else 2)) + 4), "flops": 3.0 * n}
