"""Attention over a paged cache on a GPU: scales of either sign, pages of every
size, many sequences, and work that ends anywhere."""

import numpy as np
import pytest

from tests import _gpu
from tests._gpu import torch
from tests.test_gpu_attend import check, made
from tests.test_gpu_cache import int32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0, 1e-30])
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64), ("f16", 256)])
def test_scales(tsx, scale, dtype, dim):
    att, q, cache, batch = made(tsx, dtype, 4, 2, dim, 16, [30, 1], [200, 77], spread=0.5)
    att.scale = scale
    for most in (1, 100):
        out, lse = att.forward(q, cache, batch._replace(most_new=most), lse=True)
        check(att, q, cache, batch, out, lse)


@pytest.mark.parametrize("page", [1, 3, 8, 32, 40, 64, 128, 256, 512])
@pytest.mark.parametrize("dtype,dim,order", [("bf16", 128, "slots"), ("f16", 64, "heads"), ("bf16", 72, "slots")])
def test_pages(tsx, page, dtype, dim, order):
    att, q, cache, batch = made(tsx, dtype, 6, 2, dim, page, [90, 1, 40], [700, 33, 300], order=order, seed=page)
    for most in (1, 100):
        out, lse = att.forward(q, cache, batch._replace(most_new=most), lse=True)
        check(att, q, cache, batch, out, lse)


@pytest.mark.parametrize("seqs", [32, 33, 129, 700])
@pytest.mark.parametrize("most", [1, 100])
def test_many_sequences(tsx, seqs, most):
    """As many as a warp, a block, and more; some with no new token."""
    new = [(3, 1, 0, 7)[b % 4] for b in range(seqs)]
    lengths = [n + 37 * b % 150 for b, n in enumerate(new)]
    lengths = [max(n, 1) for n in lengths]
    att, q, cache, batch = made(tsx, "bf16", 4, 2, 64, 16, new, lengths, seed=seqs)
    out = att.forward(q, cache, batch._replace(most_new=most))
    check(att, q, cache, batch, out)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("page,dim", [(24, 128), (128, 64), (8, 128)])
def test_late_values_with_other_pages(tsx, bad, page, dim):
    """As with pages of 16; the values of two keys, in the same channel and in others."""
    att, q, cache, batch = made(tsx, "bf16", 4, 1, dim, page, [300], [500])
    clean = att.forward(q, cache, batch)
    for at, ch in ((350, 3), (420, 3), (420, dim - 1)):
        cache[1][int(batch.pages[0, at // page]), at % page, 0, ch] = bad
    out = att.forward(q, cache, batch)
    assert torch.equal(out[:150], clean[:150]) and torch.isfinite(out[:150]).all()
    assert not torch.isfinite(out[150:, :, 3]).any() and not torch.isfinite(out[220:, :, dim - 1]).any()
    assert torch.equal(out[150:220, :, dim - 1], clean[150:220, :, dim - 1])
    others = [c for c in range(dim) if c not in (3, dim - 1)]
    assert torch.equal(out[..., others], clean[..., others])


def test_random_batches(tsx):
    """Sizes drawn at random: whatever runs the work is cut into, both kernels give
    what the definition says."""
    rng = np.random.default_rng(5)
    for k in range(24):
        seqs = int(rng.integers(1, 9))
        new = [int(rng.choice([0, 1, 1, 2, 17, 64, 130])) for _ in range(seqs)]
        if not sum(new):
            new[0] = 1
        lengths = [max(n + int(rng.choice([0, 1, 63, 64, 127, 128, 500])), 1) for n in new]
        hk = int(rng.choice([1, 2, 3]))
        att, q, cache, batch = made(tsx, str(rng.choice(["bf16", "f16"])), hk * int(rng.choice([1, 2, 5, 8])), hk,
                                    int(rng.choice([16, 64, 96, 128])), int(rng.choice([8, 16, 20, 64, 256])), new,
                                    lengths, seed=k, before=int(rng.integers(0, 3)), behind=int(rng.integers(0, 3)))
        for most in (1, 100):
            out, lse = att.forward(q, cache, batch._replace(most_new=most), lse=True)
            check(att, q, cache, batch, out, lse)


def test_an_empty_cache_and_no_sequences(tsx):
    att = tsx.PagedAttention("bf16", 4, 2, 64, 16)
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    none = att.new_cache(0)
    batch = tsx.Batch(int32([0, 1, 3]), int32([5, 2]), torch.zeros(2, 4, dtype=torch.int32, device="cuda"), 2)
    for most in (1, 100):
        out, lse = att.forward(q, none, batch._replace(most_new=most), lse=True)
        assert (out == 0).all() and (lse == float("-inf")).all()
    k = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(att.append(q, k, k, none, batch), q)
    # page lists of no entries
    bare = tsx.Batch(int32([0, 3]), int32([3]), torch.zeros(1, 0, dtype=torch.int32, device="cuda"), 3)
    cache = att.new_cache(2)
    for most in (1, 100):
        assert (att.forward(q, cache, bare._replace(most_new=most)) == 0).all()
    # no sequences: nothing is written
    empty = tsx.Batch(int32([0]), int32([]), torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 1)
    out = torch.full_like(q, 9)
    att.forward(q, cache, empty, out=out)
    att.append(q, k, k, cache, empty, out=out)
    assert (out == 9).all() and (cache[0] == 0).all()
