"""An attention block trained and served with the operators around attention.

Trained, queries and keys are normed and turned by one call each way (an autograd
function around ``tsx.Rotary``), and the attention itself is torch's matrix
products.  Served, a step's tokens, chunks of prompts and single ones side by side,
go into a paged cache, normed and turned on the way, and attend over it; the single
tokens' steps run from one captured CUDA graph, in whose tensors only the numbers
change::

    python examples/attention_block.py [--new 32]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import pipelined_elementwise_streaming_gb300 as tsx  # noqa: E402


class Turned(torch.autograd.Function):
    """Queries and keys normed and turned; `op` is a tsx.Rotary with a norm."""

    @staticmethod
    def forward(ctx, q, k, positions, q_weight, k_weight, op):
        ctx.save_for_backward(q, k, positions, q_weight, k_weight)
        ctx.op = op
        return op.forward(q, k, positions, q_weight, k_weight)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        q, k, positions, q_weight, k_weight = ctx.saved_tensors
        dq, dk, dq_weight, dk_weight = ctx.op.backward(dq.contiguous(), dk.contiguous(), positions, q, k, q_weight,
                                                       k_weight)
        return dq, dk, None, dq_weight, dk_weight, None


class Block(torch.nn.Module):
    def __init__(self, width: int, heads: int, kv_heads: int, dim: int, page_size: int = 16):
        super().__init__()
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.w_in = torch.nn.Parameter(torch.randn(width, (heads + 2 * kv_heads) * dim) / width**0.5)
        self.w_out = torch.nn.Parameter(torch.randn(heads * dim, width) / (heads * dim)**0.5)
        self.q_weight, self.k_weight = (torch.nn.Parameter(torch.ones(dim)) for _ in range(2))
        self.rotary = tsx.Rotary("bf16", heads, kv_heads, dim, norm="rms")
        self.attention = tsx.PagedAttention("bf16", heads, kv_heads, dim, page_size, rotary=self.rotary)

    def project(self, x):
        qkv = (x @ self.w_in.bfloat16()).view(len(x), -1, self.dim)
        return qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)

    def forward(self, x, positions):
        """One sequence x [tokens, width], each token seeing those before it."""
        q, k, v = self.project(x)
        q, k = Turned.apply(q, k, positions, self.q_weight, self.k_weight, self.rotary)
        group = self.heads // self.kv_heads
        k, v = (t.float().transpose(0, 1).repeat_interleave(group, 0) for t in (k, v))
        s = q.float().transpose(0, 1) @ k.transpose(1, 2) * self.dim**-0.5
        hidden = torch.ones(s.shape[1:], dtype=torch.bool, device=x.device).triu(1)
        y = torch.softmax(s.masked_fill(hidden, float("-inf")), -1) @ v
        return y.transpose(0, 1).flatten(1).bfloat16() @ self.w_out.bfloat16()

    @torch.no_grad()
    def step(self, x, cache, batch):
        """New tokens x of the batch's sequences, over what the cache holds of them."""
        q, k, v = self.project(x)
        q = self.attention.append(q, k, v, cache, batch, self.q_weight, self.k_weight)
        return self.attention.forward(q, cache, batch).flatten(1) @ self.w_out.bfloat16()


def serve(block: Block, prompts, new: int, chunk: int = 64, seed: int = 0):
    """The prompts [tokens, width] in chunks, then `new` tokens to each, every one
    the block's last output; all outputs of each sequence."""
    page = block.attention.page_size
    most = -(-(max(len(p) for p in prompts) + new) // page)
    seqs, device = len(prompts), prompts[0].device
    cache = block.attention.new_cache(seqs * most, device)
    order = torch.randperm(seqs * most, generator=torch.Generator().manual_seed(seed))
    pages = order.int().view(seqs, most).to(device)
    done, outs = [0] * seqs, [[] for _ in prompts]
    while any(d < len(p) for d, p in zip(done, prompts)):
        count = [min(chunk, len(p) - d) for d, p in zip(done, prompts)]
        x = torch.cat([p[d:d + n] for p, d, n in zip(prompts, done, count)])
        done = [d + n for d, n in zip(done, count)]
        starts = torch.tensor([sum(count[:b]) for b in range(seqs + 1)], dtype=torch.int32, device=device)
        lengths = torch.tensor(done, dtype=torch.int32, device=device)
        for o, y in zip(outs, block.step(x, cache, tsx.Batch(starts, lengths, pages, max(count))).split(count)):
            o.append(y)
    if not new:
        return [torch.cat(o) for o in outs]
    # single tokens: a step is captured once, its lengths and inputs change in place
    starts, lengths = torch.arange(seqs + 1, dtype=torch.int32, device=device), lengths + 1
    batch = tsx.Batch(starts, lengths, pages, 1)
    x = torch.stack([torch.cat(o)[-1] for o in outs])
    side = torch.cuda.Stream(device)
    side.wait_stream(torch.cuda.current_stream(device))
    with torch.cuda.stream(side):   # warm
        block.step(x, cache, batch)
    torch.cuda.current_stream(device).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.step(x, cache, batch)
    for _ in range(new):
        graph.replay()
        for o, row in zip(outs, y.clone()):
            o.append(row[None])
        x.copy_(y)
        lengths.add_(1)
    return [torch.cat(o) for o in outs]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--new", type=int, default=32)
    a = ap.parse_args()
    torch.manual_seed(0)
    block = Block(256, 8, 2, 64).cuda()
    prompts = [torch.randn(n, 256, device="cuda").bfloat16() for n in (100, 7, 300)]
    for b, y in enumerate(serve(block, prompts, a.new)):
        print(f"sequence {b}: {len(prompts[b])} tokens and {len(y) - len(prompts[b])} new ones, last output "
              f"{y[-1].float().norm():.3f}")
