"""Attention over a paged cache on a GPU with sums of very many weights of one
size, most of which are small against their sum."""

import pytest

from tests import _gpu
from tests._gpu import torch
from tests.test_gpu_attend import HALF_STEP

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim,group,new,most,keys", [(128, 4, 1, 1, 1 << 20), (64, 16, 1, 1, 1 << 19), (256, 2, 1, 1, 1 << 18),
                                                     (128, 12, 1, 1, 1 << 18), (128, 4, 1, 100, 1 << 20),
                                                     (64, 2, 150, 150, 1 << 18)])
@pytest.mark.parametrize("spread,climb", [(0.0, 0.0), (0.5, 0.0), (0.5, 40.0)])
def test_sums_over_very_many_keys(tsx, dtype, dim, group, new, most, keys, spread, climb):
    """The last token of sequences that are so many and so long that one block sums
    most of a sequence's keys; pages repeat, some more than others, and with
    `climb` the scores of the last pages are far above those of the first."""
    hk, seqs, page, pool = 8, 64 if new == 1 else 24, 1024, 48
    gen = torch.Generator(device="cuda").manual_seed(dim + group)
    t = _gpu.TORCH_DTYPE[dtype]
    att = tsx.PagedAttention(dtype, hk * group, hk, dim, page)
    k = torch.randn(pool, page, hk, dim, generator=gen, device="cuda")
    k[..., 0] = climb * torch.arange(pool, device="cuda")[:, None, None] / pool
    cache = k.to(t), (1 + 0.5 * torch.rand(pool, page, hk, dim, generator=gen, device="cuda")).to(t)
    q = spread * torch.randn(seqs * new, hk * group, dim, generator=gen, device="cuda")
    q[..., 0] = dim**0.5 if climb else 0.0
    q = q.to(t)
    n = keys // page
    order = (torch.rand(n, generator=gen, device="cuda").square() * pool).long().sort().values
    table = order.int().expand(seqs, n).contiguous()
    starts = (torch.arange(seqs + 1, device="cuda") * new).int()
    batch = tsx.Batch(starts, torch.full((seqs,), keys, dtype=torch.int32, device="cuda"), table, most)
    out, lse = att.forward(q, cache, batch, lse=True)
    often = torch.bincount(order, minlength=pool).double()
    for row in (new - 1, (seqs // 2) * new + new - 1, seqs * new - 1):   # last tokens see all keys
        x = torch.einsum("hgd,pshd->hgps", q[row].double().unflatten(0, (hk, group)), cache[0].double()) * att.scale
        x = (x + often.log()[:, None]).flatten(2)
        want = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), cache[1].double().flatten(0, 1)).flatten(0, 1)
        # the half steps of the result and of weights (values are positive), and what 1024 truncated additions
        # lose, 2^-23 each, and as much again in scores and exponentials
        slack = (2 * HALF_STEP[dtype] + 2.0**-12) * want
        assert ((out[row].double() - want).abs() <= slack).all()
        # lse: fp32 sums of a thread's weights, rounded to nearest, folded every 1024 of them
        assert ((lse[row].double() - torch.logsumexp(x, -1).flatten()).abs() <= 2.0**-13 + 2.0**-20 * (climb + 20)).all()
