"""Random shapes of the layer operators against their formulas in 64 bits (on
the GPU, by torch): every layout that a shape may take, odd sizes, slices and
misaligned bases among them.

Tolerances: an output rounded into its type carries half its spacing, 2^-11,
2^-8 or 2^-24 of the value; fp32 arithmetic before it, relative to the largest
value of the output, well under 2^-16 for sums of the lengths drawn (at most
2^17 terms added in a tree of short runs: errors grow with the depth, below
2^-18 of the sum of magnitudes, and the sums of magnitudes here are below four
times the largest output).  Groups of one element have the gradient zero and
xhat zero: there the kernels' differences are of equal numbers, and exact."""

import math
import random

import pytest

from tests import _gpu
from tests._gpu import torch

pytestmark = pytest.mark.gpu

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"f16": 2.0**-11, "bf16": 2.0**-8, "f32": 2.0**-24}


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


def near(got, want, dtype, what):
    got = got.double()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), what
    top = want.abs().max() if want.numel() else 0
    off = (got - want).abs() - (HALF[dtype] * 1.01 * want.abs() + 2.0**-16 * top + 2.0**-24)
    assert not off.numel() or off.max() <= 0, f"{what}: off by {off.max().item():.3g} (largest {float(top):.3g})"


def shape_of(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    g = rng.choice([1, 1, 2, 3, 8, 16, 32, 32, 57, 200])
    per = rng.choice([1, 2, 4, 5, 8, 10, 16, 24, 40, 64, 100, 128, 256]) if rng.random() < 0.7 else log(1, 3000)
    l = 1 if rng.random() < 0.15 else log(1, 20000)
    total = log(1 << 8, 1 << 20)
    n = max(1, min(3000, total // (l * g * per)))
    return n, l, g * per, g


def act64(z, kind):
    if kind == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    if kind == "gelu":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z**3))
        return z / 2 * (1 + t), (1 + t) / 2 + z / 2 * (1 - t * t) * k * (1 + 0.134145 * z * z)
    return z, torch.ones_like(z)


def put(t, dtype, pitch, shift):
    """t in rows `pitch` elements apart, its base `shift` elements into a buffer."""
    n, l, c = t.shape
    flat = torch.full((n * l * pitch + shift + 8,), float("nan"), dtype=TORCH[dtype], device="cuda")
    v = flat[shift: shift + n * l * pitch].view(n, l, pitch)[..., :c]
    v.copy_(t)
    return v


@pytest.mark.parametrize("seed", range(120))
def test_norm(tsx, seed):
    rng = random.Random(seed)
    n, l, c, g = shape_of(rng)
    dtype, act = rng.choice(["f16", "bf16", "bf16", "f32"]), rng.choice(["none", "silu", "gelu"])
    form, block = rng.choice(["int8", "e4m3"]), rng.choice([32, 64, 128])
    xp, yp = c + rng.choice([0, 0, 0, 1, 8, 24]), c + rng.choice([0, 0, 8, 3])
    sx, sy = rng.choice([0, 0, 0, 1, 8]), rng.choice([0, 0, 0, 1])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    draw = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = put(draw(n, l, c) * 1.3 + 0.4, dtype, xp, sx)
    dy = put(draw(n, l, c), dtype, yp, sy)
    w, b = 1 + 0.2 * draw(c), 0.2 * draw(c)
    what = f"{(n, l, c, g)} {dtype} {act} {form} {block} pitches {xp} {yp} bases {sx} {sy}"
    op = tsx.GroupNorm(dtype, n, l, c, g, act=act, form=form, block=block, x_pitch=xp, y_pitch=yp, eps=1e-3)

    x64 = x.double()
    v = x64.reshape(n, l, g, c // g)
    mean = v.mean((1, 3))
    var = (v - mean[:, None, :, None]).square().mean((1, 3))
    rstd = (var + 1e-3).rsqrt()
    spread = lambda t: t[:, None, :, None].expand(n, l, g, c // g).reshape(n, l, c)  # noqa: E731
    hat = (x64 - spread(mean)) * spread(rstd)
    value, slope = act64(hat * w.double() + b.double(), act)

    y, m, r, saved = op.forward(x, w, b, checkpoint=True)
    y2, m2, r2 = op.forward(x, w, b)
    for p, q, z in ((y, m, r), (y2, m2, r2)):
        near(p, value, dtype, what + " y")
        near(q, mean, "f32", what + " mean")
        near(z, rstd, "f32", what + " rstd")
    held = tsx.Packer(dtype, n * l, c, form=form, block=block).pack(x.reshape(n * l, c).contiguous())
    assert torch.equal(held.q.view(torch.int8), saved.q.view(torch.int8)) and torch.equal(held.scale, saved.scale), what

    for src, xs in ((x, x64), (saved, saved.q.double().mul_(
            saved.scale.double().repeat_interleave(block, 1)[:, :c]).reshape(n, l, c))):
        hat = (xs - spread(mean)) * spread(rstd)
        dz = dy.double() * act64(hat * w.double() + b.double(), act)[1]
        d = dz * w.double()
        group = lambda t: spread(t.reshape(n, l, g, c // g).mean((1, 3)))  # noqa: E731
        dx = spread(rstd) * (d - group(d) - hat * group(d * hat))
        got = op.backward(dy, src, w, b, m, r)
        near(got[0], dx, dtype, what + " dx")
        for k, (have, terms) in enumerate(((got[1], dz * hat), (got[2], dz))):
            scale = terms.abs().sum((0, 1)).max()
            off = (have.double() - terms.sum((0, 1))).abs().max()
            assert off <= 2.0**-16 * scale + 1e-12, (what, k, off, scale)


@pytest.mark.parametrize("seed", range(60))
def test_gated_and_checkpoints(tsx, seed):
    rng = random.Random(1000 + seed)
    rows, cols = rng.choice([1, 3, 17, 64, 333, 2000]), rng.choice([1, 8, 31, 64, 200, 1000, 2731, 4096, 11008])
    dtype, act = rng.choice(["f16", "bf16", "f32"]), rng.choice(["none", "silu", "gelu"])
    form, block = rng.choice(["int8", "e4m3"]), rng.choice([32, 64, 128])
    ip, op_ = rng.choice([cols, 2 * cols, 2 * cols + 8, 2 * cols + 1]), cols + rng.choice([0, 8, 5])
    sx = rng.choice([0, 0, 1, 8])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    draw = lambda: torch.randn(1, rows, cols, generator=gen, device="cuda")  # noqa: E731
    a, u = put(2 * draw(), dtype, ip, sx)[0], put(draw(), dtype, ip, sx)[0]
    dh = put(draw(), dtype, op_, 0)[0]
    what = f"{(rows, cols)} {dtype} {act} {form} {block} pitches {ip} {op_} base {sx}"
    f = tsx.GatedAct(dtype, rows, cols, act=act, form=form, block=block, in_pitch=ip, out_pitch=op_)
    h, ca, cu = f.forward(a, u, checkpoint=True)
    assert torch.equal(f.forward(a, u), h), what
    value, _ = act64(a.double(), act)
    near(h, value * u.double(), dtype, what + " h")
    stands = lambda s: s.q.double() * s.scale.double().repeat_interleave(block, 1)[:, :cols]  # noqa: E731
    for src, (xa, xu) in (((a, u), (a.double(), u.double())), ((ca, cu), (stands(ca), stands(cu)))):
        value, slope = act64(xa, act)
        da, du, h = f.backward(dh, *src, recompute=True)
        near(da, dh.double() * xu * slope, dtype, what + " dgate")
        near(du, dh.double() * value, dtype, what + " dup")
        near(h, value * xu, dtype, what + " h again")
    pack = tsx.Packer(dtype, rows, cols, form=form, block=block, pitch=ip)
    saved = pack.pack(a)
    assert torch.equal(saved.q.view(torch.int8), ca.q.view(torch.int8)) and torch.equal(saved.scale, ca.scale), what
    near(pack.unpack(saved), stands(saved), dtype, what + " unpacked")


def test_checkpoints_stay_in_their_buffers(tsx):
    """Bytes and scales around a checkpoint are not written, also where the
    last team of a row has no channels (6000 channels: 14 of 16 octs of its
    last block, and whole teams past it)."""
    for rows, cols, block in ((6, 6000, 128), (5, 200, 32), (3, 33, 64), (2, 2056, 128)):
        blocks = -(-cols // block)
        q = torch.full((rows * cols + 64,), 77, dtype=torch.int8, device="cuda")
        scale = torch.full((rows * blocks + 64,), -3.0, device="cuda")
        x = torch.randn(rows, cols, device="cuda").bfloat16()
        out = tsx.Checkpoint(q[32: 32 + rows * cols].view(rows, cols), scale[32: 32 + rows * blocks].view(rows, blocks))
        tsx.Packer("bf16", rows, cols, block=block).pack(x, out=out)
        want = tsx.Packer("bf16", rows, cols, block=block).pack(x)
        assert torch.equal(out.q, want.q) and torch.equal(out.scale, want.scale)
        assert (q[:32] == 77).all() and (q[32 + rows * cols:] == 77).all()
        assert (scale[:32] == -3).all() and (scale[32 + rows * blocks:] == -3).all()
