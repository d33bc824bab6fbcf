"""Attention over a paged cache on a GPU with scales and products of any size."""

import pytest

from tests import _gpu
from tests._gpu import torch
from tests.test_gpu_attend import check, made

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


@pytest.mark.parametrize("power", [-121, -100, 100, 127])
@pytest.mark.parametrize("sign", [1, -1])
def test_scales_of_any_size(tsx, power, sign):
    """Scores of ordinary size from very large and very small products."""
    att, q, cache, batch = made(tsx, "bf16", 4, 2, 64, 16, [30, 1], [200, 77], spread=0.5)
    att.scale = sign * 2.0**power
    half = -power // 2
    q *= 2.0**half
    cache = (cache[0] * 2.0 ** (-power - half), cache[1])
    for most in (1, 100):
        out, lse = att.forward(q, cache, batch._replace(most_new=most), lse=True)
        check(att, q, cache, batch, out, lse)


def test_a_scale_of_zero_and_large_products(tsx):
    """All weights alike, whatever the products are."""
    att, q, cache, batch = made(tsx, "bf16", 4, 2, 64, 16, [30, 1], [200, 77], spread=0.5)
    att.scale = 0.0
    q *= 2.0**60
    cache = (cache[0] * 2.0**60, cache[1])
    for most in (1, 100):
        out, lse = att.forward(q, cache, batch._replace(most_new=most), lse=True)
        check(att, q, cache, batch, out, lse)
