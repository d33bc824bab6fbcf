"""Attention over a paged cache on a GPU that takes longer than a wait of its
kernels is patient for: the longest sequence that there is, of pages that repeat."""

import pytest

from tests import _gpu
from tests._gpu import torch
from tests.test_gpu_cache import int32

pytestmark = pytest.mark.gpu


def test_the_longest_sequence():
    """2^31 - 2^20 keys to 12288 tokens, some seconds of work in which warps that
    bring queries wait: one key of the last page leads all others so far that each
    token's result is its value, to the bit."""
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as tsx

    page, tokens, dim = 1 << 20, 48 * 256, 8
    att = tsx.PagedAttention("bf16", 1, 1, dim, page, scale=1.0)
    cache = att.new_cache(2)
    for t in cache:
        t.fill_(7)
    q = torch.zeros(tokens, 1, dim, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    cache[0][1, 5, 0, 0] = 256
    value = torch.randn(dim, device="cuda").bfloat16()
    cache[1][1, 5, 0] = value
    table = torch.zeros(1, 2047, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    batch = tsx.Batch(int32([0, tokens]), int32([2047 * page]), table, tokens)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    out, lse = att.forward(q, cache, batch, lse=True)
    end.record()
    end.synchronize()
    print(f"{start.elapsed_time(end):.0f} ms")
    assert torch.equal(out, value.expand(tokens, 1, dim))
    assert ((lse - 256).abs() <= 256 * 2.0**-22).all()


def test_a_chunk_behind_very_long_sequences():
    """Single tokens of 64 sequences of 2^31 - 2^20, by the kernel for many rows,
    whose second tile's warps have nothing to do for seconds, and then a chunk
    that has a second tile."""
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as tsx

    page, dim, seqs, new = 1 << 20, 8, 64, 256
    att = tsx.PagedAttention("bf16", 1, 1, dim, page, scale=1.0)
    cache = att.new_cache(3)
    for t in cache:
        t.fill_(7)
    q = torch.randn(seqs + new, 1, dim, device="cuda").bfloat16()
    q[:seqs] = 0
    q[:seqs, :, 0] = 1
    cache[0][1, 5, 0, 0] = 256
    value = torch.randn(dim, device="cuda").bfloat16()
    cache[1][1, 5, 0] = value
    for t in cache:
        t[2, :300] = torch.randn(300, 1, dim, device="cuda").bfloat16()
    table = torch.zeros(seqs + 1, 2047, dtype=torch.int32, device="cuda")
    table[:, -1] = 1
    table[seqs, 0] = 2
    starts = list(range(seqs + 1)) + [seqs + new]
    batch = tsx.Batch(int32(starts), int32([2047 * page] * seqs + [300]), table, new)
    out = att.forward(q, cache, batch)
    torch.cuda.synchronize()
    assert torch.equal(out[:seqs], value.expand(seqs, 1, dim))
    alone = tsx.Batch(int32([0, new]), int32([300]), table[seqs:, :1].contiguous(), new)
    # the same steps of 128 keys: the runs may be cut elsewhere, a sum's order at most
    want = att.forward(q[seqs:].contiguous(), cache, alone).double()
    assert ((out[seqs:].double() - want).abs() <= 2.0**-7 * want.abs() + 2.0**-8 * 4).all()
