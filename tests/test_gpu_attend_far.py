"""Attention over a paged cache on a GPU whose scores are so large that fp32
numbers there lie far apart: the largest one has all the weight, and those that
tie with it share it."""

import pytest

from tests import _gpu
from tests._gpu import torch
from tests.test_gpu_attend import HALF_STEP, made

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 24)])
@pytest.mark.parametrize("power", [10, 20, 24, 27, 29, 31, 36])
@pytest.mark.parametrize("shift", [0, -11])
@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_score_has_all_the_weight(tsx, dtype, dim, page, power, shift, sign):
    """Scores are (j + shift) 2^power times 1.375, j a key's place of 11, by turns or
    climbing; all of them positive or all negative."""
    att, q, cache, batch = made(tsx, dtype, 2, 1, dim, page, [3, 1], [700, 300])
    att.scale = sign * 1.375 * 2.0 ** (power - 12)
    q[:] = 0
    q[..., 0] = sign * 2.0**10
    for b, n in enumerate(batch.lengths.tolist()):
        p = torch.arange(n, device="cuda")
        ids, slots = batch.pages[b].long()[p // page], p % page
        place = (p * 11 // n if b else p % 11)
        cache[0][ids, slots] = 0
        cache[0][ids, slots, 0, 0] = 4.0 * (place + shift).to(q.dtype)
    for most in (1, 100):
        out, lse = att.forward(q, cache, batch._replace(most_new=most), lse=True)
        for row, (b, n) in enumerate(((0, 698), (0, 699), (0, 700), (1, 300))):
            p = torch.arange(n, device="cuda")
            keys = cache[0][batch.pages[b].long()[p // page], p % page, 0, 0].double()
            best = keys == keys.max()
            v = cache[1][batch.pages[b].long()[p // page], p % page, 0].double()[best]
            want, size = v.mean(0), v.abs().mean(0)
            # the result's and the weights' half steps, and those of fp32 sums
            slack = HALF_STEP[dtype] * (want.abs() + size) + (best.sum() / 16 + 8) * 2.0**-21 * size + 1e-7
            assert ((out[row].double() - want).abs() <= slack).all()
            top = keys.max() * 1.375 * 2.0 ** (power - 2)
            # lse: the score's rounding and that of the sum of the weights' logarithm
            assert ((lse[row].double() - top - best.sum().log()).abs() <= 2.0**-21 * top.abs() + 2.0**-14).all()
