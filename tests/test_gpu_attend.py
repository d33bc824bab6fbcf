"""Attention over a paged cache on a GPU against its definition in 64 bits."""

import numpy as np
import pytest

from oracle import attention as ref
from tests import _gpu
from tests._gpu import torch
from tests.test_gpu_cache import batch_of, int32

pytestmark = pytest.mark.gpu

HALF_STEP = {"f16": 2.0**-11, "bf16": 2.0**-8}


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


def np64(t):
    return t.detach().double().cpu().numpy()


def made(tsx, dtype, hq, hk, dim, page, new, lengths, seed=0, order="slots", before=0, behind=0, spread=1.5):
    """(attention, q, cache, batch); what no sequence uses of the cache is NaN."""
    batch, pages = batch_of(tsx, new, lengths, page, seed=seed, first=before)
    att = tsx.PagedAttention(dtype, hq, hk, dim, page)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = _gpu.TORCH_DTYPE[dtype]
    q = (spread * torch.randn(before + sum(new) + behind, hq, dim, generator=gen, device="cuda")).to(t)
    cache = []
    for _ in range(2):
        shape = (pages, page, hk, dim) if order == "slots" else (pages, hk, page, dim)
        c = torch.full(shape, float("nan"), dtype=t, device="cuda")
        c = c if order == "slots" else c.transpose(1, 2)
        for b, n in enumerate(lengths):
            p = torch.arange(n, device="cuda")
            ids = batch.pages[b].long()[p // page]
            c[ids, p % page] = torch.randn(n, hk, dim, generator=gen, device="cuda").to(t)
        cache.append(c)
    return att, q, tuple(cache), batch


def check(att, q, cache, batch, out, lse=None, exclude=None):
    """out, and lse, within what the roundings give: of the result and of the
    weights half a step each; of the scores and sums what a product of matrices
    in fp32 loses, 2^-21 of the sum of magnitudes to every 16 terms."""
    q64, k, v = np64(q), np64(cache[0]), np64(cache[1])
    starts, lengths, pages = (t.cpu().numpy() for t in batch[:3])
    want, logs = ref.attend(q64, k, v, starts, lengths, pages, att.scale)
    with np.errstate(invalid="ignore"):
        size, _ = ref.attend(q64, k, np.abs(v), starts, lengths, pages, att.scale)
    longest = np.abs(np.nan_to_num(k)).max(axis=(0, 1))   # [heads, dim]
    most = np.einsum("thd,hd->th", np.abs(q64), np.repeat(longest, q.shape[1] // k.shape[2], 0)) * abs(att.scale)
    score = most * (q.shape[2] / 16 + 4) * 2.0**-21
    steps = HALF_STEP[att.dtype]
    weight = steps + 2 * score + (lengths.max() / 16 + 8) * 2.0**-21
    mine = np.array([ref.places(starts, lengths, pages, k.shape[1], k.shape[0], t) is not None for t in range(len(q))])
    got = np64(out)
    bad = ~(np.abs(got - want) <= steps * np.abs(want) * 1.01 + weight[..., None] * size + 1e-7)
    bad &= ~((got == want) | (np.isnan(got) & np.isnan(want)))   # infinities and NaN
    bad = bad[mine]
    assert not bad.any(), f"{bad.sum()} of {bad.size} values are too far off"
    if lse is not None:
        off = np.abs(np64(lse)[mine] - logs[mine])
        ok = off <= score[mine] + 2.0**-21 * (4 + np.abs(logs[mine])) + lengths.max() * 2.0**-24
        ok |= np64(lse)[mine] == logs[mine]
        assert ok.all()
    return want


SHAPES = [
    # dtype, q heads, kv heads, dim, page, order
    ("bf16", 8, 2, 128, 16, "slots"),
    ("f16", 4, 4, 64, 64, "heads"),
    ("bf16", 16, 1, 64, 7, "slots"),
    ("f16", 5, 1, 80, 24, "heads"),
    ("bf16", 6, 2, 256, 16, "slots"),
    ("f16", 2, 1, 8, 1, "slots"),
    ("bf16", 40, 2, 128, 33, "slots"),
    ("f16", 3, 3, 136, 128, "slots"),
]
BATCHES = [
    # new tokens, lengths with them, rows before and behind
    ([1], [1], 0, 0),
    ([1], [1000], 0, 0),
    ([1] * 6, [1, 63, 64, 65, 200, 17], 0, 0),
    ([5], [5], 0, 0),
    ([3, 1, 0, 70], [130, 1, 9, 70], 2, 3),
    ([257, 2], [300, 2], 0, 1),
    ([1] * 200, [1 + 3 * i % 50 for i in range(200)], 0, 0),
]


@pytest.mark.parametrize("dtype,hq,hk,dim,page,order", SHAPES)
@pytest.mark.parametrize("new,lengths,before,behind", BATCHES)
def test_values(tsx, dtype, hq, hk, dim, page, order, new, lengths, before, behind):
    """Also with NaN in every slot that no sequence uses."""
    att, q, cache, batch = made(tsx, dtype, hq, hk, dim, page, new, lengths, order=order, before=before, behind=behind)
    out = torch.full_like(q, 9.0)
    got, lse = att.forward(q, cache, batch, out=out, lse=True)
    assert got is out
    check(att, q, cache, batch, out, lse)
    first, last = before, before + sum(new)
    assert (out[:first] == 9).all() and (out[last:] == 9).all()
    # what the host believes of the new tokens changes no more than the order of sums
    for most in (1, 10**6):
        check(att, q, cache, batch, att.forward(q, cache, batch._replace(most_new=most)))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,length", [(1, 70001), (40, 30011), (1, 17)])
def test_one_sequence_by_many_blocks(tsx, dim, new, length):
    att, q, cache, batch = made(tsx, "f16", 4, 1, dim, 16, [new], [length], spread=2.5)
    out, lse = att.forward(q, cache, batch, lse=True)
    check(att, q, cache, batch, out, lse)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype,dim,hq", [("bf16", 128, 4), ("f16", 64, 1), ("bf16", 256, 2)])
@pytest.mark.parametrize("new,length", [(6, 6), (100, 260), (300, 300)])
def test_what_a_token_does_not_see_has_no_effect(tsx, bad, dtype, dim, hq, new, length):
    """An infinity or a NaN in a late key or value spoils the tokens from it on,
    as far as the definition says, and none before it."""
    att, q, cache, batch = made(tsx, dtype, hq, 1, dim, 16, [new], [length])
    clean = att.forward(q, cache, batch)
    at = length - new // 2
    page, slot = int(batch.pages[0, at // 16]), at % 16
    cache[1][page, slot, 0, 5] = bad
    out = att.forward(q, cache, batch)
    row = at - (length - new)
    assert torch.equal(out[:row], clean[:row])
    others = [c for c in range(dim) if c != 5]
    assert torch.equal(out[..., others], clean[..., others])
    want = torch.full_like(out[row:, :, 5], bad)
    assert torch.equal(out[row:, :, 5].isnan(), want.isnan()) and (bad != bad or torch.equal(out[row:, :, 5], want))
    cache[1][page, slot, 0, 5] = 0
    clean = att.forward(q, cache, batch)
    cache[0][page, slot, 0, 5] = bad
    out = att.forward(q, cache, batch)
    assert torch.equal(out[:row], clean[:row])
    if bad != bad:
        assert out[row:].isnan().all()


def test_pages_that_hold_nothing_and_rows_without_keys(tsx):
    att, q, cache, batch = made(tsx, "bf16", 4, 2, 64, 16, [1, 3, 1, 2], [100, 70, 5, 9])
    pages = batch.pages.clone()
    pages[0, 1:3] = torch.tensor([-1, 1 << 30], dtype=torch.int32)   # keys 16 .. 47 are passed over
    pages[2, 0] = -5                                                 # and all of the third sequence
    lengths = batch.lengths.clone()
    lengths[3] = 1                                                   # one of its two new tokens before its start
    held = batch._replace(pages=pages, lengths=lengths)
    for most in (1, 100):
        out, lse = att.forward(q, cache, held._replace(most_new=most), lse=True)
        check(att, q, cache, held, out, lse)
        assert (out[4] == 0).all() and (lse[4] == float("-inf")).all()
        assert (out[5] == 0).all() and (lse[5] == float("-inf")).all() and (out[6] != 0).any()
    # a length beyond the page list
    long = batch._replace(lengths=torch.full_like(batch.lengths, 0x7fffffff))
    fill = pages.clamp(0, cache[0].shape[0] - 1)
    cache = tuple(c.nan_to_num(0.5) for c in cache)
    out = att.forward(q, cache, long._replace(pages=fill))
    check(att, q, cache, long._replace(pages=fill), out)


def test_extreme_scores(tsx):
    """Scores of +-10^4 and their ties, all equal ones, and minus infinity
    everywhere."""
    att, q, cache, batch = made(tsx, "bf16", 2, 1, 64, 16, [1, 1, 1], [50, 50, 50])
    k = cache[0]
    q[:] = 0
    q[0, :, 0] = 1e3
    q[1, :, 1] = -1e3
    for b in range(3):
        p = torch.arange(50, device="cuda")
        ids = batch.pages[b].long()[p // 16]
        k[ids, p % 16, 0, 0] = (80.0 * (p % 3)).bfloat16()
        k[ids, p % 16, 0, 1] = (80.0 * (p % 5)).bfloat16()
    out, lse = att.forward(q, cache, batch, lse=True)
    check(att, q, cache, batch, out, lse)
    q[2] = 1
    for p in range(50):
        k[int(batch.pages[2, p // 16]), p % 16, 0, 3] = float("-inf")
    out, lse = att.forward(q, cache, batch, lse=True)
    assert (out[2] == 0).all() and (lse[2] == float("-inf")).all() and torch.isfinite(out[:2]).all()


def test_in_place_slices_and_head_major(tsx):
    """out over q; q a slice of a projection; q and out with heads outermost."""
    att, q, cache, batch = made(tsx, "bf16", 8, 2, 128, 16, [40, 1, 9], [400, 77, 9])
    want = att.forward(q, cache, batch)
    wide = torch.full((50, 12, 136), 7.0, dtype=q.dtype, device="cuda")
    part = wide[:, 2:10, 8:]
    part.copy_(q)
    assert att.forward(part, cache, batch, out=part) is part
    assert torch.equal(part, want)
    assert (wide[:, :2] == 7).all() and (wide[:, 10:] == 7).all() and (wide[:, :, :8] == 7).all()
    major = q.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty_like(major)
    assert torch.equal(att.forward(major, cache, batch, out=out), want)


def test_parts_join_by_their_logs(tsx):
    """One sequence's keys as two sequences': joined by lse they give the whole."""
    att, q, cache, batch = made(tsx, "f16", 4, 2, 64, 16, [1], [320])
    want = att.forward(q, cache, batch).double()
    two = tsx.Batch(int32([0, 1, 2]), int32([160, 160]), batch.pages[:, :20].reshape(2, 10).contiguous(), 1)
    out, lse = att.forward(q.repeat(2, 1, 1), cache, two, lse=True)
    w = torch.softmax(lse.double(), 0)[..., None]
    got = (w * out.double()).sum(0)
    # both sides' roundings: of parts, of the whole, and of weights
    assert ((got - want[0]).abs() <= 4 * 2.0**-11 * (out.double().abs().max() + 1)).all()


def test_a_cache_beyond_32_bits(tsx):
    """Pages at both ends of a cache of 2^32 and more elements."""
    att = tsx.PagedAttention("bf16", 4, 1, 64, 16)
    pages = (1 << 32) // (16 * 64) + 3
    whole = torch.empty(2 * pages, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
    cache = (whole[:pages], whole[pages:])
    ids = torch.tensor([0, pages - 1, pages // 2, pages - 2, 1], device="cuda")
    for c in cache:
        c[ids] = torch.randn(5, 16, 1, 64, device="cuda").bfloat16()
    small = tuple(c[ids].contiguous() for c in cache)
    k = torch.randn(3, 1, 64, device="cuda").bfloat16()
    q = torch.randn(3, 4, 64, device="cuda").bfloat16()
    for new, most in (([1, 2], 1), ([1, 2], 100)):
        starts, lengths = int32([0, 1, 3]), int32([47, 30])
        far = tsx.Batch(starts, lengths, ids[:4].int()[[0, 1, 2, 3, 1, 0]].reshape(2, 3).contiguous(), most)
        near = tsx.Batch(starts, lengths, int32([[0, 1, 2], [3, 1, 0]]), most)
        att.append(q, k, k, cache, far)
        att.append(q, k, k, small, near)
        assert torch.equal(cache[0][ids], small[0]) and torch.equal(cache[1][ids], small[1])
        assert torch.equal(att.forward(q, cache, far), att.forward(q, small, near))


def test_same_bits_again_side_by_side_and_in_a_graph(tsx):
    """Two calls at once on two streams, and a captured step whose lengths grow."""
    att, q, cache, batch = made(tsx, "bf16", 8, 2, 128, 16, [1] * 5, [900, 100, 33, 500, 64])
    many, q2, cache2, batch2 = made(tsx, "bf16", 8, 2, 128, 16, [90, 1], [900, 100], seed=1)
    want, want2 = att.forward(q, cache, batch), many.forward(q2, cache2, batch2)
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got.append((att.forward(q, cache, batch, stream=sides[0]), many.forward(q2, cache2, batch2, stream=sides[1])))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, want2) for a, b in got)
    lengths = batch.lengths.clone()
    live = batch._replace(lengths=lengths)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = att.forward(q, cache, live)
        out2 = many.forward(q2, cache2, batch2)
    for less in (0, 3, 20):
        lengths.copy_(batch.lengths - less)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, att.forward(q, cache, live)) and torch.equal(out2, want2)


@pytest.mark.parametrize("dtype,hq,hk,dim,page", [("bf16", 8, 2, 128, 16), ("f16", 4, 1, 64, 24)])
def test_serving_by_chunks_and_tokens(tsx, dtype, hq, hk, dim, page):
    """Two prompts appended in chunks of any size and then token by token, with
    norms and rotation on the way: each token's output is what attention over
    its whole sequence gives."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    t = _gpu.TORCH_DTYPE[dtype]
    rope = tsx.Rotary(dtype, hq, hk, dim, norm="rms", scaling=("yarn", 4.0, 64))
    att = tsx.PagedAttention(dtype, hq, hk, dim, page, rotary=rope)
    totals = [75, 130]
    qkv = [torch.randn(n, hq + 2 * hk, dim, generator=gen, device="cuda").to(t) for n in totals]
    w = [1 + torch.randn(dim, generator=gen, device="cuda") / 4 for _ in range(2)]
    cache = att.new_cache(40)
    each = -(-max(totals) // page)
    pages = torch.randperm(40, generator=torch.Generator().manual_seed(0))[: 2 * each].int().cuda().view(2, each)
    done, outs = [0, 0], [[], []]
    for new in ([40, 3], [1, 90], [30, 33], [1, 1], [1, 1], [1, 1], [1, 1]):
        rows = torch.cat([x[d:d + n] for x, d, n in zip(qkv, done, new)])
        done = [d + n for d, n in zip(done, new)]
        batch = tsx.Batch(int32([0, new[0], sum(new)]), int32(done), pages, max(new))
        q, k, v = rows.split([hq, hk, hk], 1)
        out = att.forward(att.append(q, k, v, cache, batch, *w), cache, batch)
        for o, part in zip(outs, out.split(new)):
            o.append(part)
    assert done == totals
    for x, o, n in zip(qkv, outs, totals):
        q, k = rope.forward(x[:, :hq], x[:, hq:hq + hk], torch.arange(n, device="cuda"), *w)
        whole = tsx.Batch(int32([0, n]), int32([n]), int32([list(range(-(-n // page)))]), n)
        flat = tuple(torch.zeros(-(-n // page) * page, hk, dim, dtype=t, device="cuda") for _ in range(2))
        flat[0][:n], flat[1][:n] = k, x[:, hq + hk:]
        check(att, q, tuple(f.view(-1, page, hk, dim) for f in flat), whole, torch.cat(o))
