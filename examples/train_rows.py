"""Trains a hashed row table with its readout, codes the rows, and reads out from the coded table.

    python examples/train_rows.py [--rows 4096] [--tokens 1024] [--steps 40]

Each token looks up `slots` rows; the readout is a root-mean-square norm of the rows side by side and an 8-bit product.
A step runs every dense operator once, forward and back:

    x      = embed_lookup(table, ids)                    rows of a batch
    y, q   = rms_norm(x)                                 with an 8-bit output
    out    = gemm_fp8(q, weight)                         the readout
    dy     = gemm_fp8(dout, weight transposed)           back through it
    dW     = gemm_fp8(dout transposed, y transposed)     in 32 bits
    dx, dg = rms_norm_grad(dy)
    rows   = embed_grad_rows(plan, dx)                   the distinct rows' gradients

Afterwards the trained rows are coded (Table.encode) and the same readout is fed from Table.lookup_decode. Data and
target are synthetic: a readout of other random rows.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import trellis_coded_row_amd as cp
import workload


class Readout:
    """norm (gain [slots d]) and product (weight [hidden, slots d])."""

    def __init__(self, width, hidden, gen):
        self.gain = torch.ones(width, device="cuda")
        self.weight = torch.randn(hidden, width, device="cuda", generator=gen) / width**0.5
        self.update()

    def update(self):
        """The 8-bit forms of the weight, which a step's products read."""
        self.w, self.ws, self.wt, self.wts = cp.quantize_fp8(self.weight, blocks=True, transposed=True)
        self.gain16 = self.gain.bfloat16()

    def forward(self, x):
        r = cp.rms_norm(x, self.gain16, fp8=True, rstd=True)
        return cp.gemm_fp8(r.q, r.scale, self.w, self.ws), r

    def backward(self, x, r, dout):
        """(dx, dweight, dgain) for the output's gradient."""
        q, s, qt, st = cp.quantize_fp8(dout, transposed=True)
        _, _, yt, yts = cp.quantize_fp8(r.y, transposed=True)
        dweight = cp.gemm_fp8(qt, st, yt, yts, dtype=torch.float32)
        dx, dgain = cp.rms_norm_grad(cp.gemm_fp8(q, s, self.wt, self.wts), x, r.rstd, self.gain16)
        return dx, dweight, dgain


def train(rows=4096, tokens=1024, slots=8, d=64, hidden=256, steps=40, rate=1.0, seed=0):
    """(losses of the steps, mean squared difference between the readouts of the trained and of the coded rows, mean
    square of the former)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, rows, (tokens * slots,), device="cuda", generator=gen)
    ids[::97] = -1  # padding: n-grams that a token lacks
    table = torch.randn(rows, d, device="cuda", generator=gen)
    readout = Readout(slots * d, hidden, gen)
    other = torch.randn(rows, d, device="cuda", generator=gen)
    target, _ = Readout(slots * d, hidden, gen).forward(
        cp.embed_lookup(other, ids, dtype=torch.bfloat16).view(tokens, slots * d))
    plan = cp.embed_plan(ids, rows)
    distinct = int(plan.count)
    losses = []
    for _ in range(steps):
        x = cp.embed_lookup(table, ids, dtype=torch.bfloat16).view(tokens, slots * d)
        out, r = readout.forward(x)
        off = out.float() - target.float()
        losses.append(off.square().mean())
        dx, dweight, dgain = readout.backward(x, r, (off / tokens).bfloat16())
        grad = cp.embed_grad_rows(plan, dx.view(-1, d))
        table.index_add_(0, plan.unique[:distinct], grad[:distinct], alpha=-rate * 100)
        readout.weight -= rate * dweight
        readout.gain -= rate * dgain
        readout.update()
    # the rows in 4 bits a step of two values, and the readout from them
    with cp.Table(rows, d, 4, workload.lut_fp16(seed)) as coded:
        coded.encode(table)
        trained, _ = readout.forward(cp.embed_lookup(table, ids, dtype=torch.bfloat16).view(tokens, slots * d))
        back = coded.lookup_decode(ids.clamp(min=0))
        back[ids < 0] = 0
        decoded, _ = readout.forward(back.view(tokens, slots * d))
        torch.cuda.synchronize()
    difference = (trained.float() - decoded.float()).square().mean()
    return [float(v) for v in losses], float(difference), float(trained.float().square().mean())


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--rows", type=int, default=4096)
    p.add_argument("--tokens", type=int, default=1024)
    p.add_argument("--steps", type=int, default=40)
    a = p.parse_args()
    losses, difference, square = train(a.rows, a.tokens, steps=a.steps)
    for k in range(0, len(losses), max(1, len(losses) // 8)):
        print(f"step {k:4d}  loss {losses[k]:.5f}")
    print(f"step {len(losses) - 1:4d}  loss {losses[-1]:.5f}")
    print(f"readout of the coded rows: mean squared difference {difference:.4f}, mean square {square:.4f}")
