"""The example's autograd functions, with plain operators in the place of the
library's."""

import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import __graft_entry__

    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class PlainNorm:
    """y = x * weight + bias stands for a norm: its gradient is as easy."""

    def forward(self, x, weight, bias):
        stats = torch.zeros(x.shape[0], 1)
        return x * weight + bias, stats, stats

    def backward(self, dy, x, weight, bias, mean, rstd):
        return dy * weight, (dy * x).sum((0, 1)), dy.sum((0, 1))


class PlainGated:
    rows, cols = 4, 3

    def forward(self, gate, up):
        return gate * up

    def backward(self, dh, gate, up, recompute):
        both = torch.cat([dh * up, dh * gate], 1)
        return both[:, : self.cols], both[:, self.cols:], gate * up


def test_gradients_and_no_second_ones(example):
    """First derivatives come through; a second one, for which the functions
    have no graph, is an error and not a part of the answer."""
    torch.manual_seed(0)
    x, weight, bias = torch.randn(4, 1, 3), torch.randn(3), torch.randn(3)
    both, out = torch.randn(4, 6), torch.randn(3, 5)
    for args, call, plain in (
            ((x, weight, bias), lambda *a: example.Norm.apply(*a, PlainNorm(), "full"), lambda x, w, b: x * w + b),
            ((both, out), lambda *a: example.Gated.apply(*a, PlainGated(), "full"),
             lambda v, o: (v[:, :3] * v[:, 3:]) @ o)):
        args = [t.requires_grad_() for t in args]
        got = torch.autograd.grad(call(*args).square().sum(), args)
        want = torch.autograd.grad(plain(*args).square().sum(), args)
        for p, q in zip(got, want):
            torch.testing.assert_close(p, q)
        first = torch.autograd.grad(call(*args).square().sum(), args, create_graph=True)
        with pytest.raises(RuntimeError, match="twice"):
            sum(t.square().sum() for t in first).backward()
