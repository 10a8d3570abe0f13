"""A layer of experts on the low-precision and expert-grouped products, trained and served:

    python -m tiled_double_buffered_amd.expert_layer [--tokens 4096] [--steps 30]

Every token goes through one expert, a two-layer network picked by a router, and through a
linear layer that all tokens share.  Training runs the experts in bfloat16 (`linear_grouped`)
and the shared layer in 8 bits (`linear_fp8`); serving holds all weights in 8 bits
(`quantize_fp8`) and answers a batch of any size, down to one token, with
`matmul_fp8_grouped` and `matmul_fp8`.  The router's logits are an FP32 product (`matmul`).
Data and initial weights are random.
"""
from __future__ import annotations

import argparse
import sys

import torch

import tiled_double_buffered_amd as tdb

BLOCK = 128


def group(experts, count):
    """(order, offsets): the tokens sorted by expert, and where each expert's begin, as the
    grouped products take them.  Nothing comes back to the host."""
    order = torch.argsort(experts, stable=True)
    sizes = (experts[:, None] == torch.arange(count, device=experts.device)).sum(0)
    offsets = torch.zeros(count + 1, dtype=torch.int32, device=experts.device)
    torch.cumsum(sizes, 0, out=offsets[1:])
    return order, offsets


class ExpertLayer:
    def __init__(self, width, hidden, experts, device, seed=0):
        g = torch.Generator(device="cpu").manual_seed(seed)

        def weights(*shape):
            w = torch.randn(*shape, generator=g) * shape[-2] ** -0.5
            return w.to(device=device, dtype=torch.bfloat16).requires_grad_()

        self.experts = experts
        self.router = torch.randn(width, experts, generator=g).to(device)
        self.w_in = weights(experts, width, hidden)
        self.w_out = weights(experts, hidden, width)
        self.shared = weights(width, width)

    def parameters(self):
        return [self.w_in, self.w_out, self.shared]

    def route(self, x):
        return group(tdb.matmul(x.float(), self.router).argmax(1), self.experts)

    def __call__(self, x):
        order, offsets = self.route(x)
        h = torch.relu(tdb.linear_grouped(x[order], self.w_in, offsets))
        y = tdb.linear_grouped(h, self.w_out, offsets)
        return torch.empty_like(x).index_copy(0, order, y) + tdb.linear_fp8(x, self.shared)

    def served(self):
        """The layer with all weights in 8 bits, one scale for each block of 128 x 128."""
        def stack(w):  # E x K x N -> E x N x K, quantized: no block spans two experts
            each = [tdb.quantize_fp8(m.t().contiguous(), (BLOCK, BLOCK)) for m in w.detach()]
            q = torch.stack([q.view(torch.uint8) for q, _ in each])
            return q.view(each[0][0].dtype), torch.stack([s for _, s in each])

        w_in, w_out = stack(self.w_in), stack(self.w_out)
        shared = tdb.quantize_fp8(self.shared.detach(), (BLOCK, BLOCK))

        def call(x):
            order, offsets = self.route(x)
            h = torch.relu(tdb.matmul_fp8_grouped(*tdb.quantize_fp8(x[order]), *w_in, offsets))
            y = tdb.matmul_fp8_grouped(*tdb.quantize_fp8(h), *w_out, offsets)
            return torch.empty_like(x).index_copy(0, order, y) + \
                tdb.matmul_fp8(*tdb.quantize_fp8(x), *shared)

        return call


def train(layer, tokens, width, steps, device, seed=1, rate=0.05):
    """Fits the layer to another of its kind, each step moving every weight by `rate` of its
    norm down its gradient; returns the loss of each step (one copy at the end) and the tokens."""
    teacher = ExpertLayer(width, layer.w_in.shape[2], layer.experts, device, seed=seed + 7)
    teacher.router = layer.router
    g = torch.Generator(device="cpu").manual_seed(seed)
    x = torch.randn(tokens, width, generator=g).to(device=device, dtype=torch.bfloat16)
    with torch.no_grad():
        target = teacher(x)
    losses = []
    for _ in range(steps):
        loss = (layer(x) - target).float().square().mean()
        grads = torch.autograd.grad(loss, layer.parameters())
        with torch.no_grad():
            for p, d in zip(layer.parameters(), grads):
                p -= rate * p.float().norm() / d.float().norm().clamp_min(1e-20) * d
        losses.append(loss.detach())
    return torch.stack(losses).tolist(), x


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args(argv)
    device = torch.device("cuda:0")
    layer = ExpertLayer(a.width, a.hidden, a.experts, device)
    losses, x = train(layer, a.tokens, a.width, a.steps, device)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    serve = layer.served()
    with torch.no_grad():
        for n in (a.tokens, 7, 1):
            y, ref = serve(x[:n]).float(), layer(x[:n]).float()
            print(f"{n} tokens served in 8 bits: {float((y - ref).norm() / ref.norm()):.4f} off "
                  "the training form")
    return 0


if __name__ == "__main__":
    sys.exit(main())
