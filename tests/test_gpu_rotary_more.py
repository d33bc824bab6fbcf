"""Gradients of head norms on a GPU where rows of threads have no head to work on."""

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
