"""A ZeRO-3 training step on virtual ranks held in one GPU's HBM, with 4-bit weights
on the wire and in the products, and 8-bit optimizer moments.

    python examples/sharded_mxfp4.py [--ranks 4] [--steps 60] [--seed 0]

A two-layer network (256 -> 512 -> 128) learns a fixed random one.  Its fp32 weights
are one flat bucket of which every rank owns an equal chunk of whole rows.  A step:

  1. every rank multiplies its own batch by the gathered weights (mxfp4_linear:
     forward and both backward products on MXFP4 payloads);
  2. the gradients are reduce-scattered with quantized hops (protocols.one_hop), which
     leaves each rank the fp32 sums of its chunk;
  3. each rank updates its chunk (adamw_step: E4M3 moments, a bf16 copy of the weights
     on the way);
  4. each rank quantizes its rows (mxfp4_quantize), the payloads are gathered, and
     every rank dequantizes them for the next step (mxfp4_dequantize).

The exchanges between virtual ranks are device-to-device copies standing in for the
collectives.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import quantized_collective_payloads_amd as qcp  # noqa: E402
from quantized_collective_payloads_amd import protocols  # noqa: E402

IN, HIDDEN, OUT, BATCH = 256, 512, 128, 96
SHAPES = [(HIDDEN, IN), (OUT, HIDDEN)]
BLOCK = 512                                       # of the gradients' INT8 payload


class Rank:
    """A rank's chunk of the flat weights: fp32, a bf16 copy, and the AdamW over the
    pieces of the matrices that fall into it."""

    def __init__(self, flat, first, count):
        self.master = flat[first:first + count].clone()
        self.copy = torch.empty(count, dtype=torch.bfloat16, device=flat.device)
        self.pieces, at = [], 0                   # (matrix, place in the chunk, rows)
        for k, (rows, cols) in enumerate(SHAPES):
            lo, hi = max(first, at), min(first + count, at + rows * cols)
            if lo < hi:
                self.pieces.append((k, lo - first, (hi - lo) // cols))
            at += rows * cols
        self.optimizer = qcp.AdamW([self.piece(self.master, p).reshape(-1) for p in self.pieces],
                                   copies=[self.piece(self.copy, p).reshape(-1) for p in self.pieces],
                                   state="e4m3", G=128)

    def piece(self, flat, p):
        k, at, rows = p
        return flat[at:at + rows * SHAPES[k][1]].view(rows, SHAPES[k][1])

    def step(self, sums, number, lr, scale):
        grads = [self.piece(sums, p).reshape(-1) for p in self.pieces]
        qcp.adamw_step(self.optimizer, grads, number, lr, weight_decay=0.0, grad_scale=scale, seed=number)

    def payloads(self):
        return [(p[0], qcp.mxfp4_quantize(self.piece(self.copy, p))) for p in self.pieces]


def gather(ranks):
    """Every rank's payload pieces, rows in order -> the bf16 weights of the products."""
    parts = [[] for _ in SHAPES]
    for r in ranks:
        for k, payload in r.payloads():
            parts[k].append(payload)
    weights = []
    for (rows, cols), p in zip(SHAPES, parts):
        codes, scales = (torch.cat([x[i] for x in p]) for i in (0, 1))
        weights.append(qcp.mxfp4_dequantize(codes, scales, cols, torch.bfloat16))
    return weights


def loss_of(weights, x, target):
    hidden = torch.nn.functional.gelu(qcp.mxfp4_linear(x, weights[0]).float()).to(torch.bfloat16)
    return (qcp.mxfp4_linear(hidden, weights[1]).float() - target).square().mean()


def train(n_ranks=4, steps=60, seed=0, log=print):
    """Returns the mean loss of every step."""
    total = sum(r * c for r, c in SHAPES)
    chunk = total // n_ranks
    if total % n_ranks or chunk % BLOCK or chunk % HIDDEN:
        raise ValueError(f"{n_ranks} ranks do not divide the weights into whole rows and blocks")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    teacher = [normal(r, c) / c ** 0.5 for r, c in SHAPES]
    flat = torch.cat([(normal(r, c) / c ** 0.5).reshape(-1) for r, c in SHAPES])
    ranks = [Rank(flat, r * chunk, chunk) for r in range(n_ranks)]
    for r in ranks:
        r.copy.copy_(r.master)
    scale = torch.full((1,), 1.0 / n_ranks, device="cuda")
    losses = []
    for number in range(1, steps + 1):
        buckets, loss = [], 0.0
        weights = [w.requires_grad_() for w in gather(ranks)]
        for _ in ranks:
            x = normal(BATCH, IN).to(torch.bfloat16)
            target = torch.nn.functional.gelu(x.float() @ teacher[0].t()) @ teacher[1].t()
            mine = loss_of(weights, x, target)
            grads = torch.autograd.grad(mine, weights)
            buckets.append(torch.cat([g.reshape(-1) for g in grads]))
            loss = loss + mine.detach()
        sums = protocols.one_hop(buckets, G=BLOCK, fmt="int8")
        for r, s in zip(ranks, sums):
            r.step(s, number, 3e-3, scale)
        losses.append(loss / n_ranks)
        if log and (number == 1 or number % 10 == 0):
            log(f"step {number:4d}  loss {losses[-1].item():.4f}", flush=True)
    return torch.stack(losses).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args()
    train(a.ranks, a.steps, a.seed)


if __name__ == "__main__":
    main()
