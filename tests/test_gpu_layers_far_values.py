"""Layer calls on values at the far ends of their types, and on tensors without
elements."""

import pytest

from tests import _gpu
from tests._gpu import torch

pytestmark = pytest.mark.gpu

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


def draw(seed, *shape, dtype="f32", scale=1.0, offset=0.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale + offset).to(TORCH[dtype])


# tokens, samples on chip (vectors, single elements), rows read twice, a group wider than a CTA's row
@pytest.mark.parametrize("n,l,c,groups", [(40, 1, 512, 8), (4, 30, 64, 8), (3, 11, 33, 3), (2, 9000, 64, 4),
                                          (2, 3, 6000, 2)])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("param", ["f32", "bf16"])
def test_channels_shut_and_held_open_by_their_bias(tsx, n, l, c, groups, act, param):
    """The slope of an activation is exactly 0 (silu, gelu) at -1e4 and
    exactly 1 at 1e4, and so it is at the type's lowest and largest number: the
    gradients agree bit for bit, and no other channel sees a difference."""
    op = tsx.GroupNorm("bf16", n, l, c, groups, act=act, param_dtype=param)
    x, dy = draw(1, n, l, c, dtype="bf16"), draw(2, n, l, c, dtype="bf16")
    w, bias = draw(3, c, scale=0.3, offset=1, dtype=param), draw(4, c, scale=0.3, dtype=param)
    far = torch.finfo(TORCH[param])

    def grads(lo, hi, held):
        b = bias.clone()
        b[1::5], b[2::7] = lo, hi
        y, mean, rstd, saved = op.forward(x, w, b, checkpoint=True)
        if act != "none":
            assert torch.all(y[..., 1::35] == 0)   # those that are not in both
        return op.backward(dy, saved if held else x, w, b, mean, rstd)

    for held in (False, True):
        for got, want in zip(grads(far.min, far.max, held), grads(-1e4, 1e4, held)):
            assert torch.isfinite(want).all()
            assert torch.equal(got, want)


@pytest.mark.parametrize("n,l,c,groups", [(3, 5, 0, 4), (700, 2, 0, 32), (3, 0, 0, 1), (0, 4, 0, 2), (5, 0, 16, 4)])
def test_statistics_of_groups_without_elements(tsx, n, l, c, groups):
    """Every output is written, whatever its memory held before."""
    x = torch.empty(n, l, c, device="cuda")
    w = torch.empty(c, device="cuda")
    op = tsx.GroupNorm("f32", n, l, c, groups, eps=1e-4)
    for _ in range(3):
        # what the allocator hands out next
        old = [torch.full((n, groups), float("nan"), device="cuda") for _ in range(8)]
        del old
        y, mean, rstd, saved = op.forward(x, w, w, checkpoint=True)
        assert y.shape == x.shape and saved.q.shape == (n * l, c)
        assert mean.shape == rstd.shape == (n, groups)
        assert torch.all(mean == 0) and torch.allclose(rstd, torch.full_like(rstd, 100.0))
        dx, dw, db = op.backward(x, x, w, w, mean, rstd)
        assert dx.shape == x.shape and torch.all(dw == 0) and torch.all(db == 0)
