"""The attention block of the examples: its gradients, and that it serves what it
was trained to."""

import importlib.util
import os

import pytest

from tests import _gpu
from tests._gpu import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    _gpu.need_gpu()
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_turned(q, k, positions, wq, wk, op):
    """The same in 64 bits by torch's autograd."""
    out = []
    f = torch.tensor(op.frequencies, dtype=torch.float64, device=q.device)
    angle = positions.double()[:, None] * f
    for x, w in ((q, wq), (k, wk)):
        x = x.double()
        x = x * (x.square().mean(-1, keepdim=True) + op.eps) ** -0.5 * w.double()
        a, b = x.chunk(2, -1)
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        out.append(torch.cat([a * c - b * s, b * c + a * s], -1))
    return out


def test_gradients(example):
    """Of a sum over the turned queries and keys: half a bf16 step of what the
    formula gives (fp32 weights' gradients 2^-16 of the sum of magnitudes), and no
    second derivative."""
    torch.manual_seed(0)
    op = example.tsx.Rotary("bf16", 4, 2, 64, norm="rms")
    q, k = (torch.randn(50, h, 64, device="cuda").bfloat16().requires_grad_() for h in (4, 2))
    w = [(1 + torch.randn(64, device="cuda") / 4).requires_grad_() for _ in range(2)]
    dq, dk = (torch.randn(50, h, 64, device="cuda").bfloat16() for h in (4, 2))
    pos = torch.arange(50, device="cuda")

    def grads(turned):
        y, z = turned(q, k, pos, *w, op)
        return torch.autograd.grad((y.double() * dq).sum() + (z.double() * dk).sum(), (q, k, *w))

    got, want = grads(example.Turned.apply), grads(plain_turned)
    for a, b in zip(got[:2], want[:2]):   # plain gradients are rounded to bf16 too: a step where both round apart
        assert ((a.double() - b.double()).abs() <= 2.0**-7 * b.double().abs() + 1e-4).all()
    for a, b, d in zip(got[2:], want[2:], (dq, dk)):
        assert ((a - b).abs() <= 2.0**-16 * 4 * d.float().abs().sum()).all()
    y, z = example.Turned.apply(q, k, pos, *w, op)
    first = torch.autograd.grad(y.float().square().sum() + z.float().square().sum(), (q, k, *w), create_graph=True)
    with pytest.raises(RuntimeError, match="twice"):
        sum(t.float().square().sum() for t in first).backward()


def test_a_training_step_runs(example):
    torch.manual_seed(0)
    block = example.Block(64, 4, 2, 32).cuda()
    x = torch.randn(40, 64, device="cuda").bfloat16()
    block(x, torch.arange(40, device="cuda")).float().square().mean().backward()
    assert all(p.grad is not None and torch.isfinite(p.grad).all() and (p.grad != 0).any() for p in block.parameters())


@pytest.mark.parametrize("heads,kv_heads,dim,page", [(8, 2, 64, 16), (4, 4, 128, 24)])
def test_serving_gives_what_the_block_computes(example, heads, kv_heads, dim, page):
    """Every output of every sequence, served in chunks and from a graph, against
    the block's own forward pass over the whole sequence."""
    torch.manual_seed(1)
    block = example.Block(96, heads, kv_heads, dim, page).cuda()
    prompts = [torch.randn(n, 96, device="cuda").bfloat16() for n in (70, 1, 133)]
    for prompt, y in zip(prompts, example.serve(block, prompts, 6)):
        assert len(y) == len(prompt) + 6
        x = torch.cat([prompt, y[len(prompt) - 1:-1]])
        with torch.no_grad():
            want = block(x, torch.arange(len(x), device="cuda"))
        # both round queries, keys, weights (served), values and the product's inputs to bf16, some 2^-8 each of the
        # values' size; a projection of heads * dim terms adds them as their root
        off = (y.float() - want.float()).abs()
        assert off.max() <= 6 * 2.0**-8 * want.float().abs().max()
