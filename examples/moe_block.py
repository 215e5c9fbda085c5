"""Token embedding, a mixture-of-experts router and its experts, together: one decoding step and one training step.

    python examples/moe_block.py [--tokens 64] [--steps 20]

The decoding step looks the tokens up, routes them and runs the experts. The training step trains the router and the
table by a loss of the routing weights alone, as a router is distilled or balanced: its gradient goes back through the
router to its matrix and to the token embeddings, whose rows are accumulated in 32 bits over micro-batches. (A loss of
the experts' output has a path through the experts too, by grouped_matmul and its gradient; not here.) Weights, tokens
and d loss / d weights are random; the router's own product is a plain matrix product and left to torch.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import primitives_device_scan_amd as ds  # noqa: E402


class Block:
    """The parameters, and the gradients that training accumulates."""

    def __init__(self, rows=32000, dim=1024, hidden=512, experts=64, top_k=6, dtype=torch.bfloat16, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std=1.0):
            return (torch.randn(shape, generator=g, device=device) * std).to(dtype)

        self.top_k, self.scale = top_k, dim ** 0.5
        self.table = normal(rows, dim, std=dim ** -0.5)
        self.router = torch.randn((dim, experts), generator=g, device=device) * dim ** -0.5
        self.w_in = normal(experts, 2 * hidden, dim, std=dim ** -0.5)
        self.w_out = normal(experts, dim, hidden, std=hidden ** -0.5)
        self.table_grad = torch.zeros((rows, dim), device=device)
        self.router_grad = torch.zeros_like(self.router)


def decode_step(block: Block, ids: torch.Tensor):
    """(x, logits, weights, chosen experts, y) of a step for the tokens `ids`."""
    x = ds.embedding(block.table, ids, scale=block.scale)
    logits = x.float() @ block.router
    weights, chosen = ds.moe_route(logits, block.top_k)
    return x, logits, weights, chosen, ds.moe_experts(x, block.w_in, block.w_out, chosen, weights)


def train_step(block: Block, ids: torch.Tensor, weight_grad: torch.Tensor):
    """Adds a micro-batch's gradients to the block's, for a loss of the routing weights with d loss / d weights =
    weight_grad [tokens, top_k]."""
    x = ds.embedding(block.table, ids, scale=block.scale)
    logits = x.float() @ block.router
    _, chosen = ds.moe_route(logits, block.top_k)
    dlogits = ds.moe_route_grad(logits, chosen, weight_grad)
    block.router_grad.addmm_(x.float().T, dlogits)
    dx = dlogits @ block.router.T
    ds.embedding_grad(dx, ids, block.table.shape[0], scale=block.scale, out=block.table_grad, accumulate=True)
    return chosen


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    block = Block()
    rows = block.table.shape[0]
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, rows, (a.tokens,), generator=g, device="cuda")
    batch = torch.randint(0, rows, (64 * a.tokens,), generator=g, device="cuda")
    wgrad = torch.randn((batch.numel(), block.top_k), generator=g, device="cuda")
    for name, step in (("decoding", lambda: decode_step(block, ids)), ("training", lambda: train_step(block, batch, wgrad))):
        step()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(a.steps):
            step()
        torch.cuda.synchronize()
        n = ids.numel() if name == "decoding" else batch.numel()
        print(f"{name}: {n} tokens a step, {(time.perf_counter() - t) / a.steps * 1e6:.1f} us a step")


if __name__ == "__main__":
    main()
