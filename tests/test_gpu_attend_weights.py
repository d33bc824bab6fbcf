"""Attention over a paged cache on a GPU where weights are of very different
sizes: one key that leads all others, and scores that climb."""

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


@pytest.mark.parametrize("dtype,dim", [("f16", 64), ("f16", 128), ("f16", 256), ("bf16", 64)])
@pytest.mark.parametrize("lead", [5.0, 10.0, 14.0, 17.0, 17.5, 20.0])
@pytest.mark.parametrize("at", [0, 7001, 16383])
def test_one_key_leads_all_others(tsx, dtype, dim, lead, at):
    """By `lead` in the exponent, and its value is 0: what is left is the sum of
    very many small weights, each of which counts."""
    att, q, cache, batch = made(tsx, dtype, 2, 1, dim, 16, [1], [16384])
    att.scale = 0.125
    gen = torch.Generator(device="cuda").manual_seed(1)
    q[:] = 0
    q[..., 0] = 8
    p = torch.arange(16384, device="cuda")
    ids, slots = batch.pages[0].long()[p // 16], p % 16
    keys = torch.zeros(16384, 1, dim, device="cuda")
    keys[:, 0, 0] = torch.rand(16384, generator=gen, device="cuda") - 0.5
    keys[at, 0, 0] = lead
    values = 0.5 + torch.rand(16384, 1, dim, generator=gen, device="cuda")
    values[at] = 0
    cache[0][ids, slots], cache[1][ids, slots] = keys.to(q.dtype), values.to(q.dtype)
    for most in (1, 100):
        out, lse = att.forward(q, cache, batch._replace(most_new=most), lse=True)
        check(att, q, cache, batch, out, lse)


@pytest.mark.parametrize("step", [0.002, 0.02])
@pytest.mark.parametrize("dim", [64, 128])
def test_scores_that_climb(tsx, dim, step):
    """Every key a little above the last: weights far above 1 until the maximum in
    use is changed, with the type's largest values."""
    att, q, cache, batch = made(tsx, "f16", 2, 1, dim, 16, [3], [4096])
    att.scale = 1.0
    q[:] = 0
    q[..., 0] = 1
    p = torch.arange(4096, device="cuda")
    ids, slots = batch.pages[0].long()[p // 16], p % 16
    cache[0][ids, slots] = 0
    cache[0][ids, slots, 0, 0] = (step * p).to(q.dtype)
    cache[1][ids, slots] = cache[1][ids, slots].clamp(-4, 4) * 16000
    for most in (1, 100):
        out, lse = att.forward(q, cache, batch._replace(most_new=most), lse=True)
        check(att, q, cache, batch, out, lse)
