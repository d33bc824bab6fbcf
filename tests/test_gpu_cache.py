"""Appending to a paged cache on a GPU: every slot of the cache and every row of
the queries against the definition, bit for bit with the rotation by itself."""

import numpy as np
import pytest

from oracle import attention as ref
from tests import _gpu
from tests._gpu import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


def int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def batch_of(tsx, new, lengths, page, spare=2, seed=0, first=0):
    """A batch with shuffled pages; entries that are not used are far out of range."""
    rng = np.random.default_rng(seed)
    each = [-(-n // page) for n in lengths]
    order = rng.permutation(sum(each) + spare)
    table = np.full((len(lengths), max(each + [1]) + 1), 0x7fffffff, np.int32)
    at = 0
    for b, n in enumerate(each):
        table[b, :n] = order[at:at + n]
        at += n
    starts = first + np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return tsx.Batch(int32(starts), int32(lengths), int32(table), max([*new, 1])), int(sum(each) + spare)


BATCHES = [
    # new tokens, lengths with them, page, rows before and behind the sequences
    ([1], [1], 16, 0, 0),
    ([1] * 5, [1, 16, 17, 40, 33], 16, 0, 0),
    ([3, 0, 1, 20], [3, 9, 65, 21], 7, 2, 3),
    ([130, 1, 64], [200, 64, 64], 64, 0, 5),
    ([2] * 1500, [2 + i % 9 for i in range(1500)], 4, 1, 1),   # more sequences than a CTA keeps
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,rot,layout,norm", [(128, 128, "half", "rms"), (64, 32, "interleaved", None),
                                                 (64, 0, "half", None), (50, 20, "half", "rms")])
@pytest.mark.parametrize("new,lengths,page,before,behind", BATCHES)
@pytest.mark.parametrize("order", ["slots", "heads"])
def test_every_slot(tsx, dtype, dim, rot, layout, norm, new, lengths, page, before, behind, order):
    hq, hk = 4, 2
    batch, pages = batch_of(tsx, new, lengths, page, first=before)
    tokens = before + sum(new) + behind
    f = tsx.Rotary(dtype, hq, hk, dim, rot=rot, layout=layout, norm=norm)
    att = tsx.PagedAttention(dtype, hq, hk, dim, page, rotary=f)
    gen = torch.Generator().manual_seed(0)
    qkv = torch.randn(tokens, hq + 2 * hk, dim, generator=gen).to(_gpu.TORCH_DTYPE[dtype]).cuda()
    q, k, v = qkv.split([hq, hk, hk], 1)
    w = [torch.randn(dim, generator=gen).cuda() for _ in range(2)] if norm else [None, None]
    if order == "slots":
        cache = tuple(t.fill_(9) for t in att.new_cache(pages))
    else:
        cache = tuple(torch.full((pages, hk, page, dim), 9.0, dtype=q.dtype, device="cuda").transpose(1, 2)
                      for _ in range(2))
    out = torch.full_like(q, 9, memory_format=torch.contiguous_format)
    att.append(q, k, v, cache, batch, *w, out=out)
    # the same rotation by itself, bit for bit
    starts, table = batch.starts.cpu().numpy(), batch.pages.cpu().numpy()
    at = [ref.places(starts, lengths, table, page, pages, t) for t in range(tokens)]
    pos = torch.tensor([p[1] if p else 0 for p in at], device="cuda")
    q2, k2 = f.forward(q, k, pos, *w)
    mine = torch.tensor([p is not None for p in at], device="cuda")
    assert torch.equal(out[mine], q2[mine]) and (out[~mine] == 9).all()
    want = [torch.full((pages, page, hk, dim), 9.0, dtype=q.dtype, device="cuda") for _ in range(2)]
    kept = [(t, p) for t, p in enumerate(at) if p]
    assert all(p[2] is not None for _, p in kept)
    rows = torch.tensor([t for t, _ in kept], device="cuda")
    ids, slots = (torch.tensor([x(p) for _, p in kept], device="cuda") for x in (lambda p: p[2], lambda p: p[1] % page))
    want[0][ids, slots], want[1][ids, slots] = k2[rows], v[rows]
    assert torch.equal(cache[0], want[0]) and torch.equal(cache[1], want[1])


def test_pages_and_lengths_out_of_range(tsx):
    """Tokens without a page, beyond their page list or before their sequence's
    start are left out; the others are stored."""
    att = tsx.PagedAttention("bf16", 2, 1, 64, 4, rotary=tsx.Rotary("bf16", 2, 1, 64))
    k = torch.ones(10, 1, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(10, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache = att.new_cache(3)
    # positions 2..5 over pages 2 and -1; a length of 99 taken for 8: positions 6, 7 on page 0; a length
    # shorter than its new tokens: positions -2..1 on page 1
    batch = tsx.Batch(int32([0, 4, 6, 10]), int32([6, 99, 2]), int32([[2, -1], [3, 0], [1, 1 << 30]]), 4)
    att.append(q, k, k, cache, batch)
    stored = (cache[1][:, :, 0, 0] != 0).cpu().numpy()
    want = np.zeros((3, 4), bool)
    want[2, 2:] = want[0, 2:] = want[1, :2] = True
    assert (stored == want).all()


def test_keys_alone_and_a_captured_step(tsx):
    """q None: only keys and values; a graph that is replayed with new numbers
    in the batch's tensors."""
    f = tsx.Rotary("bf16", 4, 2, 64)
    att = tsx.PagedAttention("bf16", 4, 2, 64, 8, rotary=f)
    q, k, v = (torch.randn(3, h, 64, device="cuda").bfloat16() for h in (4, 2, 2))
    cache, plain = att.new_cache(9), att.new_cache(9)
    batch = tsx.Batch(int32([0, 1, 2, 3]), int32([1, 7, 8]), int32([[0, 1], [2, 3], [4, 5]]), 1)
    assert att.append(None, k, v, plain, batch) is None
    att.append(q, k, v, cache, batch)
    assert torch.equal(cache[0], plain[0]) and torch.equal(cache[1], plain[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = att.append(q, k, v, cache, batch)
    for _ in range(3):
        batch.lengths.add_(1)
        graph.replay()
        want = att.append(q, k, v, plain, batch)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(cache[0], plain[0]) and torch.equal(cache[1], plain[1])
