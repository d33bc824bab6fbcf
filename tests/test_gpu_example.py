"""The example block: trains from 8-bit checkpoints as it does from the saved
tensors, and its gradients are near autograd's own."""

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
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_training_falls_alike(example):
    full = example.train(30, "full")
    assert full[-1] < 0.5 * full[0]
    for saved in ("int8", "e4m3"):
        # the same data and start: the first loss is the same, later ones differ by the checkpoints' rounding
        losses = example.train(30, saved)
        assert losses[0] == full[0]
        assert losses[-1] < 1.1 * full[-1]


def test_gradients_against_autograd(example):
    """The block in elementary fp32 operations: bf16 products and roundings
    leave a few 2^-8 of the gradients' size, int8 checkpoints half a step of
    1 / 127 of a block's largest value, e4m3 2^-4 of each value, averaged over
    512 channels or more."""
    tokens, width, heads, hidden = 256, 512, 8, 1024
    for saved, most in (("full", 0.02), ("int8", 0.03), ("e4m3", 0.06)):
        torch.manual_seed(1)
        block = example.Block(tokens, width, heads, hidden, saved).cuda()
        x = torch.randn(tokens, width, device="cuda", dtype=torch.bfloat16)
        dy = torch.randn(tokens, width, device="cuda")
        (block(x).float() * dy).sum().backward()
        got = [p.grad.float() for p in block.parameters()]
        w = [p.detach().clone().requires_grad_() for p in block.parameters()]
        v = x.float().reshape(tokens, heads, -1)
        hat = ((v - v.mean(-1, keepdim=True)) / (v.var(-1, unbiased=False, keepdim=True) + 1e-5).sqrt()).reshape(
            tokens, width)
        both = (hat * w[0] + w[1]) @ w[2]
        gate, up = both[:, :hidden], both[:, hidden:]
        y = x.float() + (gate * torch.sigmoid(gate) * up) @ w[3]
        (y * dy).sum().backward()
        for a, b in zip(got, w):
            assert (a - b.grad).norm() <= most * b.grad.norm(), saved
