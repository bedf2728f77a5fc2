"""An expert layer trained and served with the library's operators.

    python examples/expert_layer.py

Tokens are routed to two of the experts each, sorted by expert, and run through
y = relu(x W1 + b1) W2 (grouped_matmul, bias and ReLU in its epilogue).  The
backward pass is the input gradient (grouped_matmul with the transposed weights)
and the weight gradients (grouped_weight_grad), the update an orthogonalised
momentum (orthogonalize) of every expert's matrices at once.  The trained
weights are then rounded to 4 bits (quantize_q4) and single tokens served with
q4_matmul.  The layer learns to imitate another expert layer with fixed random
weights; routing, loss and token bookkeeping are plain torch.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_epilogues_gb300 as G  # noqa: E402

TOP = 2   # experts per token


def route(x, router):
    """(offsets, order, weight): rows sorted by expert, each row's token, and its
    share of the token's output.  Nothing waits for the host."""
    share, expert = torch.softmax(x.float() @ router, -1).topk(TOP, -1)
    expert, order = expert.flatten().sort(stable=True)
    offsets = torch.zeros(router.shape[1] + 1, dtype=torch.int32, device=x.device)
    offsets[1:] = torch.bincount(expert, minlength=router.shape[1]).cumsum(0)
    return offsets, order // TOP, (share / share.sum(-1, keepdim=True)).flatten()[order]


class Experts:
    """E experts of width d -> h -> d, bf16 weights with fp32 momentum."""

    def __init__(self, experts, d, h, seed, device="cuda"):
        gen = torch.Generator(device).manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=gen, device=device)   # noqa: E731
        self.w1 = (rand(experts, d, h) * d ** -0.5).bfloat16()
        self.b1 = torch.zeros((experts, h), device=device)
        self.w2 = (rand(experts, h, d) * h ** -0.5).bfloat16()
        self.plan = G.Plan(G.GEMM_BF16, G.GEMM_F32, torch.cuda.current_device())
        self.plan32 = G.Plan(G.GEMM_F32, G.GEMM_F32, torch.cuda.current_device())
        self.momentum = [torch.zeros_like(w, dtype=torch.float32) for w in (self.w1, self.w2)]

    def forward(self, x, offsets):
        """Rows of x (sorted by expert) -> (y, the hidden rows)."""
        h = G.grouped_matmul(x, self.w1, offsets, bias=self.b1, relu=True, plan=self.plan)
        return G.grouped_matmul(h, self.w2, offsets, plan=self.plan), h

    def backward(self, x, h, dy, offsets):
        """Gradients of W1 and W2 (fp32) for the rows' output gradient dy."""
        dw2 = G.grouped_weight_grad(h, dy, offsets, out_dtype=torch.float32, plan=self.plan)
        dh = G.grouped_matmul(dy, self.w2.transpose(1, 2), offsets, plan=self.plan)
        dh *= h > 0
        return G.grouped_weight_grad(x, dh, offsets, out_dtype=torch.float32, plan=self.plan), dw2

    def update(self, grads, rate, beta=0.9):
        """Each expert's matrices move along their orthogonalised momentum."""
        for w, m, g in zip((self.w1, self.w2), self.momentum, grads):
            m.mul_(beta).add_(g)
            step = G.orthogonalize(m, plan=self.plan32)
            w.sub_(step, alpha=rate * max(1.0, w.shape[1] / w.shape[2]) ** 0.5)

    def quantised(self, group=64):
        """4-bit weights of both products, [experts, N, K / 2] packed along K."""
        return [G.quantize_q4(w.transpose(1, 2).contiguous(), group, zero_points=True) for w in (self.w1, self.w2)]


def serve_q4(x, offsets, packed, b1, group, plan):
    (q1, s1, z1), (q2, s2, z2) = packed
    h = G.q4_matmul(x, q1, s1, group, zeros=z1, offsets=offsets, bias=b1, relu=True, plan=plan)
    return G.q4_matmul(h, q2, s2, group, zeros=z2, offsets=offsets, plan=plan)


def combine(y, order, weight, tokens):
    out = torch.zeros((tokens, y.shape[1]), device=y.device)
    return out.index_add_(0, order, y.float() * weight[:, None])


def main(experts=8, d=256, h=512, tokens=1024, steps=60, rate=0.02, group=64, seed=0, verbose=True):
    gen = torch.Generator("cuda").manual_seed(seed)
    router = torch.randn((d, experts), generator=gen, device="cuda") * d ** -0.5
    teacher, student = Experts(experts, d, h, seed + 1), Experts(experts, d, h, seed + 2)
    losses = []
    for step in range(steps):
        x = torch.randn((tokens, d), generator=gen, device="cuda").bfloat16()
        offsets, order, weight = route(x, router)
        rows = x[order]
        target = combine(teacher.forward(rows, offsets)[0], order, weight, tokens)
        y, hidden = student.forward(rows, offsets)
        error = combine(y, order, weight, tokens) - target
        losses.append(float(error.square().mean()))
        dy = (error[order] * weight[:, None] * (2.0 / error.numel())).bfloat16()
        student.update(student.backward(rows, hidden, dy, offsets), rate * (1 - step / steps))
        if verbose and step % 10 == 0:
            print(f"step {step:3d}  loss {losses[-1]:.4f}")
    # One token at a time, with 4-bit weights.
    packed = student.quantised(group)
    worst = 0.0
    for _ in range(4):
        x = torch.randn((1, d), generator=gen, device="cuda").bfloat16()
        offsets, order, weight = route(x, router)
        rows = x[order]
        full = combine(student.forward(rows, offsets)[0], order, weight, 1)
        low = combine(serve_q4(rows, offsets, packed, student.b1, group, student.plan), order, weight, 1)
        worst = max(worst, float((low - full).norm() / full.norm()))
    if verbose:
        print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; 4-bit weights change an output by {100 * worst:.1f} % at most")
    assert student.plan.device_status() == 0 and student.plan32.device_status() == 0
    return losses, worst


if __name__ == "__main__":
    main()
