"""Attention over a paged cache on a GPU where weights are of very different
sizes: one key that leads all others, scores that climb, and what is lost of
weights; and infinite values that have weight."""

import numpy as np
import pytest

from oracle import attention as ref
from tests import _gpu
from tests._gpu import torch
from tests.test_gpu_attend import HALF_STEP, check, made, np64

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


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("bf16", 64), ("bf16", 256), ("f16", 64), ("f16", 128), ("f16", 200)])
@pytest.mark.parametrize("hq,hk,new,most", [(8, 1, [1, 1], 1), (6, 3, [4, 1], 4), (4, 2, [1, 30], 1)])
def test_weights_of_up_to_eight_rows_lose_no_half_step(tsx, dtype, dim, hq, hk, new, most):
    """Where a head has up to 8 rows (or is taken to have), only the result is
    rounded to the element type: weights are good to 2^-16 (bf16) or 2^-22."""
    att, q, cache, batch = made(tsx, dtype, hq, hk, dim, 16, new, [190, 77], spread=0.5)
    batch = batch._replace(most_new=most)
    got = np64(att.forward(q, cache, batch))
    q64, k, v = np64(q), np64(cache[0]), np64(cache[1])
    starts, lengths, pages = (t.cpu().numpy() for t in batch[:3])
    want, _ = ref.attend(q64, k, v, starts, lengths, pages, att.scale)
    size, _ = ref.attend(q64, k, np.abs(v), starts, lengths, pages, att.scale)
    keys = np.repeat(np.linalg.norm(np.nan_to_num(k), axis=-1).max((0, 1)), hq // hk)
    # scores: dim / 16 additions of 16 products in fp32, each to 2^-21 of the products' magnitudes
    score = np.linalg.norm(q64, axis=-1) * keys * att.scale * (dim / 16 + 4) * 2.0**-21
    rest = {"bf16": 2.0**-16, "f16": 2.0**-22}[dtype]
    slack = HALF_STEP[dtype] * np.abs(want) * 1.01 + (rest + 2 * score + (190 / 16 + 8) * 2.0**-21)[..., None] * size
    assert (np.abs(got - want) <= slack + 2.0**-25).all()


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64), ("bf16", 256)])
@pytest.mark.parametrize("hq", [1, 8, 16])
@pytest.mark.parametrize("most", [1, 100])
def test_infinities_that_every_row_sees(tsx, dtype, dim, hq, most):
    """In values of an early key: infinite results, NaN where both signs meet, and
    other channels as they were."""
    att, q, cache, batch = made(tsx, dtype, hq, 1, dim, 16, [2, 1], [300, 290], spread=0.5)
    batch = batch._replace(most_new=most)
    want = att.forward(q, cache, batch)
    inf = float("inf")
    for at, channel, bad in ((3, 0, inf), (100, 1, -inf), (7, 2, inf), (250, 2, -inf), (64, dim - 1, inf), (90, dim - 1, inf)):
        cache[1][int(batch.pages[0, at // 16]), at % 16, 0, channel] = bad
    for channel, value in ((0, inf), (1, -inf), (2, float("nan")), (dim - 1, inf)):
        want[:2, :, channel] = value
    out = att.forward(q, cache, batch)
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out.nan_to_num(9.0, 1e4, -1e4), want.nan_to_num(9.0, 1e4, -1e4))
