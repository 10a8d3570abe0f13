"""A layer of experts on the low-precision and expert-grouped products, trained and served:

    python -m tiled_double_buffered_amd.expert_layer [--tokens 4096] [--steps 30] [--top 2]

Every token goes through one expert, a two-layer network picked by a router, and through a
linear layer that all tokens share.  Training runs the experts in bfloat16 (`linear_grouped`)
and the shared layer in 8 bits (`linear_fp8`); serving holds all weights in 8 bits
(`quantize_fp8`) and answers a batch of any size, down to one token, with
`matmul_fp8_grouped` and `matmul_fp8`.  The router's logits are an FP32 product (`matmul`).

With --top K every token goes through K gated experts of a router that is trained with them
(`RoutedLayer`): `route_experts` gives its gates and a balance loss, `group_rows` the rows by expert;
`linear_grouped` and `gated_silu` keep what their backward passes need in 8 bits.  Beside the shared
linear layer stand adapters of low rank (`add_adapters`), one for each request, trained and served.
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


class RoutedLayer:
    """`top` gated experts for every token, from a trained router, and a shared linear layer with an
    adapter for each request.  x: tokens x width; requests: the adapter of each token, or -1; valid:
    False for padding, whose result is the shared layer's alone."""

    def __init__(self, width, hidden, experts, device, top=2, adapters=4, rank=16, seed=0,
                 dtype=torch.bfloat16, checkpoint=True):
        g = torch.Generator(device="cpu").manual_seed(seed)

        def weights(*shape, scale=None, dtype=dtype):
            w = torch.randn(*shape, generator=g) * (shape[-2] ** -0.5 if scale is None else scale)
            return w.to(device=device, dtype=dtype).requires_grad_()

        self.experts, self.adapters, self.top, self.checkpoint = experts, adapters, top, checkpoint
        self.router = weights(1, width, experts, dtype=torch.float32)
        self.w_in = weights(experts, width, 2 * hidden)   # gate's columns, then up's
        self.w_out = weights(experts, hidden, width)
        self.shared = weights(width, width)
        self.down = weights(adapters, rank, width, scale=width ** -0.5)
        self.up = weights(adapters, rank, width, scale=0.1 * rank ** -0.5)

    def parameters(self):
        return [self.router, self.w_in, self.w_out, self.shared, self.down, self.up]

    def _route(self, x, valid):
        rows = torch.arange(2, dtype=torch.int32, device=x.device) * x.shape[0]  # one "expert"
        logits = tdb.linear_grouped(x.float(), self.router, rows)
        gates, experts, _, loss = tdb.route_experts(logits, self.top, valid=valid, renormalize=True)
        return gates, tdb.group_rows(experts, self.experts), loss

    @staticmethod
    def _join(y, place, gates):
        return (y[place] * gates[..., None].to(y.dtype)).sum(1)

    def __call__(self, x, requests, valid=None):
        """(y, the router's balance loss)"""
        gates, (order, place, offsets), loss = self._route(x, valid)
        h = tdb.linear_grouped(x[order // self.top], self.w_in, offsets, checkpoint=self.checkpoint)
        h = tdb.gated_silu(h, checkpoint=self.checkpoint)
        y = tdb.linear_grouped(h, self.w_out, offsets, checkpoint=self.checkpoint)
        order, _, offsets = tdb.group_rows(requests, self.adapters)
        base = tdb.linear_fp8(x, self.shared)
        base = tdb.add_adapters(base, x, self.down, self.up, order, offsets)
        return self._join(y, place, gates) + base, loss

    def served(self):
        """The layer with its weights in 8 bits (the adapters as they are)."""
        def stack(w):
            each = [tdb.quantize_fp8(m.t().contiguous(), (BLOCK, BLOCK)) for m in w.detach()]
            q = torch.stack([q.view(torch.uint8) for q, _ in each])
            return q.view(each[0][0].dtype), torch.stack([s for _, s in each])

        w_in, w_out = stack(self.w_in), stack(self.w_out)
        shared = tdb.quantize_fp8(self.shared.detach(), (BLOCK, BLOCK))
        dtype = self.shared.dtype

        def call(x, requests, valid=None):
            gates, (order, place, offsets), _ = self._route(x, valid)
            h = tdb.matmul_fp8_grouped(*tdb.quantize_fp8(x[order // self.top]), *w_in, offsets, dtype)
            y = tdb.matmul_fp8_grouped(*tdb.quantize_fp8(tdb.gated_silu(h)), *w_out, offsets, dtype)
            order, _, offsets = tdb.group_rows(requests, self.adapters)
            base = tdb.matmul_fp8(*tdb.quantize_fp8(x), *shared, dtype)
            base = tdb.add_adapters(base, x, self.down, self.up, order, offsets)
            return self._join(y, place, gates) + base

        return call


def train_routed(layer, tokens, width, steps, device, seed=1, rate=0.05, balance=0.01):
    """Fits a RoutedLayer to another of its kind, as `train` does, a tenth of the tokens padding and
    as many without an adapter; returns the loss and the balance loss of each step, the tokens and
    their requests."""
    teacher = RoutedLayer(width, layer.w_out.shape[1], layer.experts, device, layer.top,
                          layer.adapters, layer.down.shape[1], seed=seed + 7,
                          dtype=layer.shared.dtype, checkpoint=layer.checkpoint)
    g = torch.Generator(device="cpu").manual_seed(seed)
    x = torch.randn(tokens, width, generator=g).to(device=device, dtype=layer.shared.dtype)
    requests = torch.randint(0, layer.adapters, (tokens,), generator=g).to(device)
    requests[::10] = -1
    valid = torch.arange(tokens, device=device) % 10 != 5
    with torch.no_grad():
        target = teacher(x, requests, valid)[0]
    losses = []
    for _ in range(steps):
        y, even = layer(x, requests, valid)
        loss = (y - target).float().square().mean()
        grads = torch.autograd.grad(loss + balance * even, layer.parameters())
        with torch.no_grad():
            for p, d in zip(layer.parameters(), grads):
                p -= rate * p.float().norm() / d.float().norm().clamp_min(1e-20) * d
        losses.append(torch.stack([loss.detach(), even.detach()]))
    return torch.stack(losses).tolist(), x, requests


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
    ap.add_argument("--top", type=int, default=0, help="experts of a token, with a trained router")
    a = ap.parse_args(argv)
    device = torch.device("cuda:0")
    if a.top:
        layer = RoutedLayer(a.width, a.hidden, a.experts, device, top=a.top)
        losses, x, requests = train_routed(layer, a.tokens, a.width, a.steps, device)
        print(f"loss {losses[0][0]:.4f} -> {losses[-1][0]:.4f}, balance {losses[0][1]:.4f} -> "
              f"{losses[-1][1]:.4f} in {a.steps} steps")
        serve = layer.served()
        with torch.no_grad():
            for n in (a.tokens, 7, 1):
                y = serve(x[:n], requests[:n]).float()
                ref = layer(x[:n], requests[:n])[0].float()
                print(f"{n} tokens served in 8 bits: {float((y - ref).norm() / ref.norm()):.4f} off "
                      "the training form")
        return 0
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
