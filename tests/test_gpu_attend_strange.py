"""Values that are not finite in batches of many short sequences, where a block
goes over many tiles: they reach the tokens that see them, and no other
sequence's."""

import pytest

from tests import _gpu
from tests._gpu import torch
from tests.test_gpu_attend import made

pytestmark = pytest.mark.gpu

# New tokens of the sequences by turns, two queries to a key: tiles of a few rows one
# after the other, and with tiles of more than 128 rows among them.
SHORT = (1, 3, 17, 1, 64)
MIXED = (1, 90, 5, 200, 1, 1, 64)


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


@pytest.mark.parametrize("turns", [SHORT, MIXED], ids=["short", "mixed"])
@pytest.mark.parametrize("dtype,dim,page", [("bf16", 128, 16), ("f16", 64, 16), ("bf16", 64, 24), ("f16", 128, 24)])
@pytest.mark.parametrize("most", [1, 100])
def test_strange_values_of_one_sequence_stay_its_own(tsx, turns, dtype, dim, page, most):
    seqs, hk = 400, 3
    new = [turns[b % len(turns)] for b in range(seqs)]
    lengths = [n + 31 * b % 170 for b, n in enumerate(new)]
    att, q, cache, batch = made(tsx, dtype, 2 * hk, hk, dim, page, new, lengths, seed=dim + page)
    batch = batch._replace(most_new=most)
    clean = att.forward(q, cache, batch)
    assert torch.isfinite(clean).all()
    held = cache[1].clone()
    starts, pages = batch.starts.tolist(), batch.pages.tolist()
    for first in range(3):   # which sequences have one, and what
        cache[1].copy_(held)
        want = clean.clone()
        for b in range(first, seqs, 3):
            bad = (float("nan"), float("inf"), float("-inf"))[b // 3 % 3]
            row = new[b] // 2 if b % 2 else new[b] - 1   # the first new token that sees it
            at, head, channel = lengths[b] - new[b] + row, b % hk, 7 * b % dim
            cache[1][pages[b][at // page], at % page, head, channel] = bad
            want[starts[b] + row:starts[b + 1], 2 * head:2 * head + 2, channel] = bad
        for _ in range(4):
            out = att.forward(q, cache, batch)
            assert torch.equal(out.isnan(), want.isnan())
            assert torch.equal(out.nan_to_num(9.0, 1e4, -1e4), want.nan_to_num(9.0, 1e4, -1e4))
