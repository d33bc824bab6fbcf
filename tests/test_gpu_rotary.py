"""Rotary positions and norms of heads on a GPU against their definitions in 64
bits, at the layouts, sizes and positions where they can go wrong."""

import numpy as np
import pytest

from oracle import attention as ref
from tests import _gpu
from tests._gpu import torch

pytestmark = pytest.mark.gpu

HALF_STEP = {"f16": 2.0**-11, "bf16": 2.0**-8, "f32": 2.0**-24}
LEAST = {"f16": 2.0**-25, "bf16": 2.0**-126, "f32": 2.0**-126}
# Sines and cosines: under 2^-22 (fp32), 2^-19 (16 bits), a product and an fma on
# top (2^-23 of either term); a norm's sum of squares, root and two products stay
# under 2^-20 in all.
TURNED = {"f16": 2.0**-18, "bf16": 2.0**-18, "f32": 2.0**-20}


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


def made(shape, dtype, seed, extra=0, order="tokens"):
    """A tensor [tokens, heads, dim], a slice of one that is `extra` wider in
    every dimension, or with its heads outermost."""
    gen = torch.Generator().manual_seed(seed)
    tokens, heads, dim = shape
    wide = (tokens, heads + (1 if extra else 0), dim + extra)
    x = torch.randn(wide, generator=gen) * torch.exp(torch.randn(wide[-1], generator=gen) / 2)
    x = x.to(_gpu.TORCH_DTYPE[dtype]).cuda()
    if order == "heads":
        x = x.transpose(0, 1).contiguous().transpose(0, 1)
    return x[:, :heads, extra // 2:extra // 2 + dim]


def positions(tokens, far, seed, dtype=None):
    gen = torch.Generator().manual_seed(seed)
    return torch.randint(-far // 8, far, (tokens,), generator=gen).to(dtype or torch.int64).cuda()


def np64(t):
    return t.detach().double().cpu().numpy()


def reach(x, rot, layout):
    """|a| + |b| of each channel's pair, |x| of the others."""
    out = np.abs(x)
    a, b = ref.pairs(rot, layout)
    both = out[..., a] + out[..., b]
    out[..., a], out[..., b] = both, both
    return out


def near(got, want, slack, what):
    off = np.abs(np64(got) - want) - slack
    assert not np.isnan(off).any() and (off <= 0).all(), \
        f"{what}: {int((off > 0).sum())} of {off.size} values are too far off, the worst by {off.max():.3g} more"


CASES = [
    # tokens, q heads, k heads, dim, rot, layout, extra, order, far, scaling
    (1, 1, 1, 128, 128, "half", 0, "tokens", 1 << 20, None),
    (7, 32, 8, 128, 128, "half", 0, "tokens", 1 << 20, ("yarn", 16.0, 32768)),
    (1, 5, 0, 64, 64, "interleaved", 0, "tokens", 100, None),
    (3, 0, 2, 64, 32, "half", 0, "tokens", 100, None),
    (130, 12, 12, 64, 64, "half", 0, "tokens", 4096, ("linear", 4.0)),
    (2000, 9, 3, 96, 64, "interleaved", 8, "tokens", 4096, ("ntk", 4.0)),
    (2000, 9, 3, 96, 64, "half", 16, "tokens", 4096, ("ntk", 4.0)),
    (333, 6, 2, 72, 40, "interleaved", 0, "heads", 1 << 30, None),
    (33, 4, 4, 256, 256, "half", 8, "heads", 1 << 30, None),
    (33, 4, 4, 256, 8, "interleaved", 0, "tokens", 1 << 16, None),
    (17, 3, 1, 8, 8, "interleaved", 0, "tokens", 1 << 16, None),
    (17, 3, 1, 16, 16, "half", 0, "tokens", 1 << 16, None),
    (65, 3, 1, 80, 80, "half", 0, "tokens", 1 << 16, None),
    # element by element: odd sizes, a rot without whole octs, pitches of single elements
    (19, 3, 2, 1, 0, "half", 0, "tokens", 100, None),
    (19, 3, 2, 2, 2, "half", 0, "tokens", 100, None),
    (70, 5, 2, 75, 50, "half", 0, "tokens", 4096, None),
    (70, 5, 2, 75, 74, "interleaved", 3, "tokens", 4096, None),
    (41, 2, 1, 128, 24, "half", 0, "tokens", 4096, None),
    (41, 3, 1, 128, 128, "half", 2, "heads", 4096, None),
    (41, 2, 3, 255, 254, "interleaved", 1, "tokens", 4096, None),
    (5, 2, 2, 64, 0, "half", 0, "tokens", 4096, None),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot,layout,extra,order,far,scaling", CASES)
def test_values_and_gradients(tsx, dtype, tokens, hq, hk, dim, rot, layout, extra, order, far, scaling):
    freq, amp = ref.frequencies(rot, scaling=scaling)
    for norm in (None, "rms"):
        f = tsx.Rotary(dtype, hq, hk, dim, rot=rot, layout=layout, scaling=scaling, norm=norm, eps=1e-3)
        pos = positions(tokens, far, 3, torch.int32 if tokens % 2 else torch.int64)
        x = [made((tokens, h, dim), dtype, 5 + i, extra, order) if h else None for i, h in enumerate((hq, hk))]
        d = [made((tokens, h, dim), dtype, 7 + i, extra, order) if h else None for i, h in enumerate((hq, hk))]
        gen = torch.Generator().manual_seed(1)
        w = [(1 + torch.randn(dim, generator=gen) / 4).cuda() if norm and h else None for h in (hq, hk)]
        held = [t.clone() if t is not None else None for t in x + d]
        y = f.forward(*x, pos, *w)
        grads = f.backward(*d, pos, *(x if norm else (None, None)), *w)
        p64 = pos.cpu().numpy()
        k = TURNED[dtype]
        for i, h in enumerate((hq, hk)):
            if not h:
                assert y[i] is None and grads[i] is None
                continue
            x64, d64 = np64(x[i]), np64(d[i])
            w64 = np64(w[i]) if norm else np.ones(dim)
            normed = ref.norm(x64, w64, 1e-3)[0] if norm else x64
            want = ref.turn(normed, p64, freq, amp, layout)
            near(y[i], want, HALF_STEP[dtype] * np.abs(want) * (1 + 2**-8) + k * amp * reach(normed, rot, layout)
                 + LEAST[dtype], f"forward {i} {norm}")
            back = ref.turn(d64, p64, freq, amp, layout, back=True)
            size = amp * reach(d64, rot, layout)
            if not norm:
                near(grads[i], back, HALF_STEP[dtype] * np.abs(back) * (1 + 2**-8) + k * size + LEAST[dtype],
                     f"backward {i}")
                continue
            dx, dw = ref.norm_backward(back, x64, w64, 1e-3)
            _, hat, rstd = ref.norm(x64, w64, 1e-3)
            # d's error, the norm's of xhat and rstd twice over, the mean's sum
            terms = rstd * (size * np.abs(w64) + np.abs(hat) * (size * np.abs(w64 * hat)).mean(-1, keepdims=True))
            near(grads[i], dx, HALF_STEP[dtype] * np.abs(dx) * (1 + 2**-8) + 4 * k * terms + LEAST[dtype],
                 f"backward {i}")
            total = (size * np.abs(hat)).sum((0, 1))
            near(grads[2 + i], dw, (2 * k + (tokens * h + 40) * 2.0**-24) * total + 1e-30, f"dweight {i}")
        assert all(a is None or torch.equal(a, b) for a, b in zip(x + d, held))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 50])
def test_gradient_against_differences(tsx, dtype, dim):
    """Of sum(dy y) in directions of the weights and of the inputs: central
    differences of the definition in 64 bits."""
    tokens, hq, hk, rot, eps = 9, 3, 2, 32, 1e-3
    f = tsx.Rotary(dtype, hq, hk, dim, rot=rot, norm="rms", eps=eps)
    freq, amp = ref.frequencies(rot)
    pos = positions(tokens, 1000, 1)
    q, k, dq, dk = (made((tokens, h, dim), dtype, s) for s, h in enumerate((hq, hk, hq, hk)))
    wq, wk = (torch.randn(dim, generator=torch.Generator().manual_seed(s)).cuda() for s in (5, 6))
    gq, gk, gwq, gwk = f.backward(dq, dk, pos, q, k, wq, wk)
    for x, w, d, gx, gw in ((q, wq, dq, gq, gwq), (k, wk, dk, gk, gwk)):
        x, w, d = np64(x), np64(w), np64(d)

        def loss(x, w):
            return (d * ref.turn(ref.norm(x, w, eps)[0], pos.cpu().numpy(), freq, amp, "half")).sum()

        rng = np.random.default_rng(0)
        u, z, t = rng.standard_normal(x.shape), rng.standard_normal(w.shape), 1e-6
        along = (loss(x + t * u, w) - loss(x - t * u, w)) / (2 * t)
        # each gradient within its half step, and 1e-6 for the differences
        assert abs(along - (u * np64(gx)).sum()) <= (HALF_STEP[dtype] + 1e-6) * np.abs(u * np64(gx)).sum() + 1e-5
        along = (loss(x, w + t * z) - loss(x, w - t * z)) / (2 * t)
        assert abs(along - (z * np64(gw)).sum()) <= 2e-4 * np.abs(z * np64(gw)).sum() + 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 64), (50, 20)])
def test_what_does_not_turn_is_kept_and_nothing_else_is_written(tsx, dtype, dim, rot):
    """Channels beyond rot keep their bits, infinities and NaN in them stay
    theirs; in place; between the rows nothing changes."""
    tokens, heads = 37, 3
    for layout in ("half", "interleaved"):
        f = tsx.Rotary(dtype, heads, heads, dim, rot=rot, layout=layout)
        whole = torch.full((tokens, heads + 1, dim + 8), 7.0, dtype=_gpu.TORCH_DTYPE[dtype], device="cuda")
        q = whole[:, :heads, :dim]
        q.copy_(made((tokens, heads, dim), dtype, 2))
        if rot < dim:
            q[3, 1, rot], q[3, 1, rot + 1], q[4, 0, dim - 1] = float("inf"), float("nan"), float("-inf")
        k = q.clone()
        before = q.clone()
        pos = positions(tokens, 5000, 4)
        want = f.forward(q, k, pos)
        f.forward(q, k, pos, q_out=q, k_out=k)
        bits = torch.int32 if dtype == "f32" else torch.int16
        for got in (q, k):
            assert torch.equal(got.contiguous().view(bits), want[0].view(bits))
        assert torch.equal(q[..., rot:].contiguous().view(bits), before[..., rot:].contiguous().view(bits))
        assert torch.isfinite(q[..., :rot]).all()
        assert (whole[:, heads] == 7).all() and (whole[:, :, dim:] == 7).all()


def test_a_turn_and_back(tsx):
    """Far positions: the gradient's rotation undoes the first, and positions
    that a whole number of 2^64ths apart turn alike."""
    f = tsx.Rotary("f32", 2, 2, 64)
    q = made((6, 2, 64), "f32", 1)
    pos = torch.tensor([0, 1, -1, 2**31, -(2**40), 2**62], device="cuda")
    y, _ = f.forward(q, q, pos)
    assert torch.equal(y[0], q[0])
    back, _ = f.backward(y, y, pos)
    # two rotations of an error of 2^-20 each
    assert ((back - q).abs().cpu().numpy() <= 2.0**-18 * reach(np64(q), 64, "half")).all()
    # exact angles at 2^62 and -2^40: thousandths of a turn in whole numbers
    turns = list(f._desc.turns[:32])
    for row, p in ((4, -(2**40)), (5, 2**62)):
        angle = np.array([(t * p) % 2**64 / 2**64 * 2 * np.pi for t in turns])
        x = np64(q)[row]
        want = x[:, :32] * np.cos(angle) - x[:, 32:] * np.sin(angle)
        assert (np.abs(np64(y)[row, :, :32] - want) <= 2.0**-20 * reach(np64(q)[row], 64, "half")[:, :32]).all()


def test_rows_of_zeros_and_far_values(tsx):
    f = tsx.Rotary("bf16", 1, 1, 64, norm="rms", eps=1e-6)
    w = torch.ones(64, device="cuda")
    x = torch.zeros(5, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[1] = 1e18
    x[2] = 1e-18
    x[3, 0, 5] = float("nan")
    x[4] = 1.0
    pos = torch.zeros(5, dtype=torch.int64, device="cuda")
    y, _ = f.forward(x, x, pos, w, w)
    assert (y[0] == 0).all() and (y[1] == 1).all() and (y[4] == 1).all()
    assert torch.isnan(y[3]).all() and torch.isfinite(y[2]).all()
    dx, _, dw, _ = f.backward(torch.ones_like(x), torch.ones_like(x), pos, x, x, w, w)
    assert (dx[0].float() - 1000).abs().max() <= 4   # 1 / sqrt(1e-6)
    assert torch.isnan(dx[3]).all() and torch.isfinite(dx[[0, 1, 2, 4]]).all() and torch.isnan(dw[5])


@pytest.mark.parametrize("param_dtype", ["f32", "bf16"])
def test_weights_of_either_type_and_one_missing(tsx, param_dtype):
    f = tsx.Rotary("bf16", 4, 2, 64, norm="rms", param_dtype=param_dtype)
    t = _gpu.TORCH_DTYPE[param_dtype]
    wq = (1 + torch.arange(64, device="cuda") / 64).to(t)
    off = torch.ones(65, dtype=t, device="cuda")[1:] * 2   # off 16 bytes
    q, k = made((50, 4, 64), "bf16", 1), made((50, 2, 64), "bf16", 2)
    pos = positions(50, 99, 0)
    y, z = f.forward(q, k, pos, wq, None)
    plain = tsx.Rotary("bf16", 4, 2, 64, norm="rms")
    ones = torch.ones(64, device="cuda")
    a, b = plain.forward(q, k, pos, wq.float(), ones)
    assert torch.equal(y, a) and torch.equal(z, b)
    got = f.backward(q, k, pos, q, k, wq, None)
    want = plain.backward(q, k, pos, q, k, wq.float(), ones)
    assert got[3] is None and all(torch.equal(p, r) for p, r in zip(got[:3], want[:3]))
    assert torch.equal(f.forward(q, k, pos, off, None)[0], plain.forward(q, k, pos, off.float(), None)[0])


def test_no_tokens(tsx):
    f = tsx.Rotary("bf16", 4, 2, 64, norm="rms")
    q, k = (torch.empty(0, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    w = torch.ones(64, device="cuda")
    pos = torch.empty(0, dtype=torch.int64, device="cuda")
    y, z = f.forward(q, k, pos, w, w)
    assert y.shape == q.shape and z.shape == k.shape
    *_, gq, gk = f.backward(q, k, pos, q, k, w, w)
    assert (gq == 0).all() and (gk == 0).all()


def test_same_bits_again_on_other_streams_and_in_a_graph(tsx):
    f = tsx.Rotary("bf16", 16, 4, 128, norm="rms")
    q, k, dq, dk = (made((3000, h, 128), "bf16", i) for i, h in enumerate((16, 4, 16, 4)))
    w = torch.rand(128, device="cuda") + 0.5
    pos = positions(3000, 9999, 0)

    def both(stream=None):
        return (*f.forward(q, k, pos, w, w, stream=stream), *f.backward(dq, dk, pos, q, k, w, w, stream=stream))

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for t in held:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))
