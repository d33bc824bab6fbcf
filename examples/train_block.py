"""A feed-forward block trained with the layer operators, its activations saved
in 8 bits for the backward pass.

One block: heads of the residual stream normalised (group norm over tokens), a
projection to gate and up side by side, the gated activation, a projection
back, the residual.  Torch's autograd runs it: two autograd functions wrap the
operators' forward and backward calls, and keep checkpoints (or, for
comparison, the tensors themselves).  The gradients have no gradients of their
own: a second derivative is an error::

    python examples/train_block.py [--steps 60] [--saved int8|e4m3|full]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import pipelined_elementwise_streaming_gb300 as tsx  # noqa: E402


class Norm(torch.autograd.Function):
    """act(group norm of x [n, l, c]); `op` is a tsx.GroupNorm."""

    @staticmethod
    def forward(ctx, x, weight, bias, op, saved):
        if saved == "full":
            y, mean, rstd = op.forward(x, weight, bias)
            held = (x,)
        else:
            y, mean, rstd, held = op.forward(x, weight, bias, checkpoint=True)
        ctx.save_for_backward(weight, bias, mean, rstd, *held)
        ctx.op = op
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        weight, bias, mean, rstd, *held = ctx.saved_tensors
        src = held[0] if len(held) == 1 else tsx.Checkpoint(*held)
        dx, dweight, dbias = ctx.op.backward(dy.contiguous(), src, weight, bias, mean, rstd)
        return dx, dweight, dbias, None, None


class Gated(torch.autograd.Function):
    """act(gate) * up for the halves of both [rows, 2 * cols], followed by the
    product with `out` [cols, c]: h is not kept, the backward pass forms it
    again for the product's weight gradient.  `op` is a tsx.GatedAct with
    in_pitch 2 * cols."""

    @staticmethod
    def forward(ctx, both, out, op, saved):
        gate, up = both[:, : op.cols], both[:, op.cols:]
        if saved == "full":
            h, held = op.forward(gate, up), (both,)
        else:
            h, a, b = op.forward(gate, up, checkpoint=True)
            held = (*a, *b)
        ctx.save_for_backward(out, *held)
        ctx.op = op
        return h @ out

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        out, *held = ctx.saved_tensors
        op = ctx.op
        if len(held) == 1:
            src = held[0][:, : op.cols], held[0][:, op.cols:]
        else:
            src = tsx.Checkpoint(*held[:2]), tsx.Checkpoint(*held[2:])
        dgate, _, h = op.backward((dy @ out.t()).contiguous(), *src, recompute=True)
        # dgate and dup are the halves of one tensor
        dboth = dgate.as_strided((op.rows, 2 * op.cols), (2 * op.cols, 1))
        return dboth, h.t() @ dy, None, None


class Block(torch.nn.Module):
    def __init__(self, tokens: int, width: int, heads: int, hidden: int, saved: str):
        super().__init__()
        form = "int8" if saved == "full" else saved
        self.saved = saved
        self.weight, self.bias = (torch.nn.Parameter(f(width)) for f in (torch.ones, torch.zeros))
        self.w_in = torch.nn.Parameter(torch.randn(width, 2 * hidden) / width**0.5)
        self.w_out = torch.nn.Parameter(torch.randn(hidden, width) / hidden**0.5)
        self.norm = tsx.GroupNorm("bf16", tokens, 1, width, heads, form=form)
        self.gated = tsx.GatedAct("bf16", tokens, hidden, act="silu", in_pitch=2 * hidden, form=form)

    def forward(self, x):
        y = Norm.apply(x[:, None], self.weight, self.bias, self.norm, self.saved)[:, 0]
        both = y @ self.w_in.bfloat16()
        return x + Gated.apply(both, self.w_out.bfloat16(), self.gated, self.saved)


def train(steps: int = 60, saved: str = "int8", tokens: int = 1024, width: int = 512, heads: int = 8,
          hidden: int = 1024, seed: int = 0, log=None):
    """Losses of `steps` steps that fit the block to a fixed random map."""
    torch.manual_seed(seed)
    block = Block(tokens, width, heads, hidden, saved).cuda()
    target = (torch.randn(width, width) / width**0.5).cuda()
    opt = torch.optim.Adam(block.parameters(), lr=4e-3)
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, width, device="cuda")
        opt.zero_grad(set_to_none=True)
        loss = (block(x.bfloat16()).float() - x @ target).square().mean()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
        if log and step % 10 == 0:
            log(f"step {step:3d}  loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--saved", choices=["int8", "e4m3", "full"], default="int8")
    a = ap.parse_args()
    print(f"last loss {train(a.steps, a.saved, log=print)[-1]:.4f}")
