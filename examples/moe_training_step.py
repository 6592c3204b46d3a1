"""Training steps of a mixture-of-experts layer whose exchanges are compressed,
on one GPU: several ranks' batches run one after another, and what ranks would
send each other goes through ``compress`` and back.

A step of a rank:
  route -> plan -> dispatch -> [all-to-all] -> experts -> [all-to-all] -> combine
and backwards, then for the ranks together
  gradients -> [reduce-scatter] -> AdamW -> [all-gather] -> parameters
Every [exchange] is a compressed one.  Attention and the layer's gate are left to
torch, and so are the experts' products, or they run in 8-bit floating point
(--fp8): then no chunk size is needed on the host for them.

    python examples/moe_training_step.py --steps 20 [--fp8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lossless_bf16_tensor_zipccl_gb300 as zc  # noqa: E402


class Sent:
    """Bytes that the exchanges took, plain and compressed."""
    plain = packed = 0


def exchange(x, chunk_elems):
    """What arrives of a bfloat16 tensor sent chunk by chunk: the same bits."""
    c = zc.compress(x, chunk_elems)
    Sent.plain += 2 * c.n
    Sent.packed += c.nbytes()
    return zc.decompress(c).view(x.shape)


class Layer:
    """Gate and experts: float32 parameters with bfloat16 copies, one flat
    buffer, and AdamW states in 8 (or 32) bits."""

    def __init__(self, hidden, experts, bits, seed=0, fp8=False):
        self.fp8 = fp8
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.experts, self.bits, self.steps = hidden, experts, bits, 0
        shapes = [(experts, hidden), (experts, hidden, hidden)]
        sizes = [torch.Size(s).numel() for s in shapes]
        flat = torch.randn(sum(sizes), generator=g, device="cuda") * hidden ** -0.5
        self.flat, self.copy = flat, flat.bfloat16()
        self.gate, self.up = (t.view(s) for t, s in zip(self.copy.split(sizes), shapes))
        self.param, self.copies = list(flat.split(sizes)), list(self.copy.split(sizes))
        self.sizes = sizes
        self.states = [zc.adamw_state(p, bits) for p in self.param]

    def forward_backward(self, x, target, top_k):
        """One rank's batch: its loss and the gradient of the flat parameters."""
        tokens, hidden = x.shape
        logits = x @ self.gate.T
        weights, ids = zc.moe_route(logits, top_k)
        plan = zc.moe_plan(ids, self.experts)
        rows = zc.moe_dispatch(x, plan.slots)
        counts = plan.counts.tolist()                    # chunk sizes: the host has to know what to send
        used = sum(counts)
        chunks = [c * hidden for c in counts]
        arrived = exchange(rows[:used], chunks)          # all-to-all: tokens to their experts
        out = torch.zeros_like(rows)
        pieces = arrived.split(counts)
        if self.fp8:
            in_rows, in_columns = zc.moe_quantize_columns(arrived, plan.offsets, by_rows=True)
            matrices = zc.moe_quantize_weights(self.up.mT.contiguous())
            zc.moe_matmul(in_rows, matrices, plan.offsets, out=out[:used])
        else:
            for e, (a, o) in enumerate(zip(pieces, out[:used].split(counts))):
                torch.matmul(a, self.up[e], out=o)
        out[:used] = exchange(out[:used], chunks)        # all-to-all: and back
        y = zc.moe_combine(out, plan.slots, weights, residual=x)

        loss = (y.float() - target).square().mean()
        grad_y = ((y.float() - target) * (2.0 / y.numel())).bfloat16()
        grad_out, grad_weights = zc.moe_combine_backward(grad_y, out, plan.slots, weights)
        grad_out = exchange(grad_out[:used], chunks)
        if self.fp8:
            grad_columns = zc.moe_quantize_columns(grad_out, plan.offsets)
            grad_up = zc.moe_matmul_backward_weights(grad_columns, in_columns, plan.offsets).mT
        else:
            grad_up = torch.stack([a.T @ g for a, g in zip(pieces, grad_out.split(counts))])
        grad_logits = zc.moe_route_backward(grad_weights, logits, ids)
        grad_gate = grad_logits.T @ x
        return loss, torch.cat([grad_gate.reshape(-1), grad_up.reshape(-1)]).bfloat16()

    def update(self, grads, lr):
        """The ranks' gradients summed, and one step of the parameters."""
        sent = [zc.compress(g) for g in grads]
        Sent.plain += sum(2 * c.n for c in sent)
        Sent.packed += sum(c.nbytes() for c in sent)
        total = zc.decompress_reduce([c.chunk(0) for c in sent], self.flat.numel())   # reduce-scatter, receiving end
        mean = torch.full((1,), 1.0 / len(grads), device="cuda")
        self.steps += 1
        m, v = [s[0] for s in self.states], [s[1] for s in self.states]
        scales = ([s[2] for s in self.states], [s[3] for s in self.states]) if self.bits == 8 else None
        zc.adamw_step(self.param, list(total.split(self.sizes)), m, v, step=self.steps, lr=lr, weight_decay=0.0,
                      scales=scales, copies=self.copies, grad_scale=mean)
        self.copy.copy_(exchange(self.copy, [self.copy.numel()]))                     # all-gather of the parameters


def train(steps=20, ranks=4, tokens=2048, hidden=512, experts=16, top_k=2, bits=8, lr=2e-3, seed=1, fp8=False):
    """Losses of `steps` steps on a fixed synthetic task, and the exchanges' compression ratio."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    layer = Layer(hidden, experts, bits, fp8=fp8)
    mix = torch.randn(hidden, hidden, generator=g, device="cuda") * hidden ** -0.5
    batches = [torch.randn(tokens, hidden, generator=g, device="cuda") for _ in range(ranks)]
    targets = [x + (x @ mix).relu() for x in batches]
    Sent.plain = Sent.packed = 0
    losses = []
    for _ in range(steps):
        done = [layer.forward_backward(x.bfloat16(), t, top_k) for x, t in zip(batches, targets)]
        layer.update([g for _, g in done], lr)
        losses.append(sum(float(l) for l, _ in done) / ranks)
    return losses, Sent.packed / Sent.plain


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("steps", 20), ("ranks", 4), ("tokens", 2048), ("hidden", 512), ("experts", 16), ("top-k", 2),
                        ("bits", 8)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--lr", type=float, default=2e-3)
    ap.add_argument("--fp8", action="store_true", help="the experts' products in 8-bit floating point")
    losses, ratio = train(**{k.replace("-", "_"): v for k, v in vars(ap.parse_args()).items()})
    for i, loss in enumerate(losses):
        print(f"step {i:3d}  loss {loss:.5f}")
    print(f"the exchanges took {100 * ratio:.1f}% of their plain bytes")


if __name__ == "__main__":
    main()
