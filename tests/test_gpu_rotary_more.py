"""Gradients of head norms on a GPU where threads have no head to work on, and of
very many tokens."""

import numpy as np
import pytest

from oracle import attention as ref
from tests import _gpu
from tests._gpu import torch
from tests.test_gpu_rotary import HALF_STEP, LEAST, TURNED, made, near, np64, positions, reach

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot", [(1, 1, 1, 128, 128), (7, 3, 1, 64, 32), (3, 5, 2, 72, 40),
                                                  (2001, 9, 3, 96, 96), (41, 3, 1, 50, 20)])
def test_gradients_without_eps(tsx, dtype, tokens, hq, hk, dim, rot):
    """eps 0: a norm's root of what a thread without a head holds is that of 0."""
    f = tsx.Rotary(dtype, hq, hk, dim, rot=rot, norm="rms", eps=0.0)
    freq, amp = ref.frequencies(rot)
    pos = positions(tokens, 4096, 3)
    x = [made((tokens, h, dim), dtype, 5 + i) for i, h in enumerate((hq, hk))]
    d = [made((tokens, h, dim), dtype, 7 + i) for i, h in enumerate((hq, hk))]
    gen = torch.Generator().manual_seed(1)
    w = [(1 + torch.randn(dim, generator=gen) / 4).cuda() for _ in range(2)]
    grads = f.backward(*d, pos, *x, *w)
    k = TURNED[dtype]
    for i, h in enumerate((hq, hk)):
        x64, d64, w64 = np64(x[i]), np64(d[i]), np64(w[i])
        back = ref.turn(d64, pos.cpu().numpy(), freq, amp, "half", back=True)
        dx, dw = ref.norm_backward(back, x64, w64, 0.0)
        _, hat, rstd = ref.norm(x64, w64, 0.0)
        # as with an eps: d's error, the norm's of xhat and rstd twice over, the mean's sum
        size = amp * reach(d64, rot, "half")
        terms = rstd * (size * np.abs(w64) + np.abs(hat) * (size * np.abs(w64 * hat)).mean(-1, keepdims=True))
        near(grads[i], dx, HALF_STEP[dtype] * np.abs(dx) * (1 + 2**-8) + 4 * k * terms + LEAST[dtype], f"backward {i}")
        total = (size * np.abs(hat)).sum((0, 1))
        near(grads[2 + i], dw, (2 * k + (tokens * h + 40) * 2.0**-24) * total + 1e-30, f"dweight {i}")


def weight_gradient64(f, dy, x, pos):
    """(the weight's gradient, the sum of magnitudes that its roundings are relative
    to) in 64 bits on the device, of heads in halves with an rms norm."""
    freq = torch.tensor(f.frequencies, dtype=torch.float64, device="cuda")
    dw, total = (torch.zeros(x.shape[-1], dtype=torch.float64, device="cuda") for _ in range(2))
    for at in range(0, len(x), 1 << 14):
        part = slice(at, at + (1 << 14))
        angle = pos[part].double()[:, None, None] * freq
        d, h = dy[part].double(), x[part].double()
        hat = h * (h.square().mean(-1, keepdim=True) + f.eps).rsqrt()
        a, b = d.chunk(2, -1)
        c, s = angle.cos(), angle.sin()
        back = torch.cat([a * c + b * s, b * c - a * s], -1)
        reach = (a.abs() + b.abs()).repeat(1, 1, 2)
        dw += (back * hat).sum((0, 1))
        total += (reach * hat.abs()).sum((0, 1))
    return dw, total


@pytest.mark.parametrize("dtype,dim,heads", [("bf16", 8, 1), ("f16", 128, 3), ("f32", 20, 2), ("f32", 64, 5)])
def test_weights_gradients_of_very_many_tokens(tsx, dtype, dim, heads):
    """300001 tokens, each block staying for many rounds of them; all terms of the
    sum have one sign, so that a round left out or taken twice shows."""
    n = 300001
    f = tsx.Rotary(dtype, heads, 0, dim, norm="rms")
    gen = torch.Generator(device="cuda").manual_seed(dim)
    x = torch.randn(n, heads, dim, generator=gen, device="cuda").to(_gpu.TORCH_DTYPE[dtype])
    w = 0.5 + torch.rand(dim, generator=gen, device="cuda")
    pos = torch.randint(1 << 20, (n,), generator=gen, device="cuda")
    y, _ = f.forward(x, None, pos, w)
    _, _, dw, _ = f.backward(y, None, pos, x, None, w)
    want, total = weight_gradient64(f, y, x, pos)
    assert (want > 0.4 * n * heads).all()
    # A thread adds 200 heads at most (900003 over 304 blocks of 16 teams, 600002 over 456 of 8 warps), then lanes,
    # warps and blocks 64 sums more; each term as in the tests of few tokens
    assert ((dw.double() - want).abs() <= (2 * TURNED[dtype] + 264 * 2.0**-24) * total).all()
