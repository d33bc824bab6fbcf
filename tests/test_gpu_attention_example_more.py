"""The weights' gradients of the attention block of the examples, channel by
channel."""

import pytest

from tests import _gpu
from tests._gpu import torch
from tests.test_gpu_attention_example import example, plain_turned  # noqa: F401
from tests.test_gpu_rotary import TURNED
from tests.test_gpu_rotary_more import weight_gradient64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 50, 700])
def test_gradients_of_weights(example, tokens):  # noqa: F811
    """Each channel's within the roundings of the terms that its sum adds."""
    torch.manual_seed(0)
    op = example.tsx.Rotary("bf16", 4, 2, 64, norm="rms")
    q, k, dq, dk = (torch.randn(tokens, h, 64, device="cuda").bfloat16() for h in (4, 2, 4, 2))
    q.requires_grad_(), k.requires_grad_()
    w = [(1 + torch.randn(64, device="cuda") / 4).requires_grad_() for _ in range(2)]
    pos = torch.arange(tokens, device="cuda")

    def grads(turned):
        y, z = turned(q, k, pos, *w, op)
        return torch.autograd.grad((y.double() * dq).sum() + (z.double() * dk).sum(), w)

    got, want = grads(example.Turned.apply), grads(plain_turned)
    for a, b, x, d in zip(got, want, (q, k), (dq, dk)):
        by_formula, total = weight_gradient64(op, d, x.detach(), pos)
        assert ((b.double() - by_formula).abs() <= 2.0**-23 * total).all()   # torch's is rounded to fp32
        assert ((a - b).abs() <= (2 * TURNED["bf16"] + (4 * tokens + 64) * 2.0**-24) * total).all()
