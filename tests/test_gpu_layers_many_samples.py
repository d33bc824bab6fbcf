"""The gradient of a group norm over so many samples that each CTA adds up
several of them for dweight and dbias (sums of more than 16 MB otherwise),
against the formula in 64 bits.

Tolerances: dx carries half its type's spacing, and fp32 arithmetic over groups
of at most 2^15 terms added in a tree of short runs, under 2^-18 of the sum of
magnitudes, which is below four times the largest value: 2^-16 of that.  A
channel's sum over samples and rows passes through fewer than 256 additions
(at most 64 rows of a lane, 32 lanes, 30 samples of a CTA, 40 slices of a
thread, 6 of a warp and 32 warps), each within 2^-24 of the sum of magnitudes:
2^-16 of that."""

import ctypes

import pytest

from tests import _gpu
from tests._gpu import torch

pytestmark = pytest.mark.gpu

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"f16": 2.0**-11, "bf16": 2.0**-8, "f32": 2.0**-24}

# n, l, c, groups.  Samples on chip: eight channels within a group, and not; single elements.  Rows read twice:
# groups wider than a CTA's row, vectors and not; samples that no CTA holds, all three.
SHAPES = [(8192, 1, 1024, 1), (3001, 2, 1024, 8), (4096, 1, 1992, 166), (4096, 1, 1001, 7),
          (1500, 1, 4096, 1), (701, 3, 4099, 1), (2200, 32, 1000, 1), (1100, 32, 2008, 2), (2200, 32, 1001, 1)]


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


def draw(seed, *shape, dtype="f32", scale=1.0, offset=0.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale + offset).to(TORCH[dtype])


def gradient(dy, x, w, b, mean, rstd, groups):
    """(dx, terms of dweight, terms of dbias) with silu, in 64 bits"""
    n, l, c = x.shape
    spread = lambda t: t.double()[:, None, :, None].expand(n, l, groups, c // groups).reshape(n, l, c)  # noqa: E731
    over = lambda t: spread(t.reshape(n, l, groups, c // groups).mean((1, 3)))  # noqa: E731
    hat = (x - spread(mean)) * spread(rstd)
    z = hat * w.double() + b.double()
    p = torch.sigmoid(z)
    dz = dy.double() * p * (1 + z * (1 - p))
    d = dz * w.double()
    return spread(rstd) * (d - over(d) - hat * over(d * hat)), dz * hat, dz


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_gradient(tsx, shape, dtype):
    n, l, c, groups = shape
    op = tsx.GroupNorm(dtype, n, l, c, groups, act="silu", eps=1e-3)
    need = op._scratch[1][0]
    assert need <= (16 << 20) + 8 * groups * n * 3
    x, dy = draw(1, n, l, c, dtype=dtype, scale=1.3, offset=0.4), draw(2, n, l, c, dtype=dtype)
    w, b = draw(3, c, scale=0.2, offset=1), draw(4, c, scale=0.2)
    _, mean, rstd, saved = op.forward(x, w, b, checkpoint=True)
    stands = (saved.q.double() * saved.scale.double().repeat_interleave(128, 1)[:, :c]).reshape(n, l, c)
    for src, values in ((x, x.double()), (saved, stands)):
        dx, t_w, t_b = gradient(dy, values, w, b, mean, rstd, groups)
        got = op.backward(dy, src, w, b, mean, rstd)
        most = HALF[dtype] * 1.01 * dx.abs() + 2.0**-16 * dx.abs().max() + 2.0**-24
        off = (got[0].double() - dx).abs() - most
        assert torch.isfinite(got[0]).all() and off.max() <= 0
        for have, terms in ((got[1], t_w), (got[2], t_b)):
            off = (have.double() - terms.sum((0, 1))).abs() - 2.0**-16 * terms.abs().sum((0, 1))
            assert off.max() <= 0
        del dx, t_w, t_b, most, off
        # again, in place, and with a scratch of exactly the size that was asked for
        again = dy.clone()
        assert all(torch.equal(p, q) for p, q in zip(op.backward(again, src, w, b, mean, rstd, out=again), got))
        buffer = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
        held = (src.data_ptr(), None, None) if torch.is_tensor(src) else (None, *(t.data_ptr() for t in src))
        rest = [t.data_ptr() for t in (w, b, mean, rstd, *out, buffer)]
        rc = tsx.tsx_group_norm_backward(ctypes.byref(op._desc), dy.data_ptr(), *held, *rest, need,
                                         torch.cuda.current_stream().cuda_stream)
        assert rc == tsx.TSX_OK, tsx.tsx_last_error()
        assert all(torch.equal(p, q) for p, q in zip(out, got))
        assert torch.all(buffer[need:] == 0xA5)


def test_the_last_samples_of_uneven_shares(tsx):
    """Samples whose number is no multiple of the CTAs': dy is zero but in the
    first and the last sample, so that their sums alone show."""
    for n, l, c, groups in ((4097, 1, 1024, 1), (1499, 1, 4096, 1), (4095, 1, 1001, 7)):
        op = tsx.GroupNorm("f32", n, l, c, groups)
        x, dy = draw(5, n, l, c), torch.zeros(n, l, c, device="cuda")
        dy[0], dy[-1] = 1.0, 2.0
        w, b = draw(6, c, scale=0.2, offset=1), draw(7, c, scale=0.2)
        _, mean, rstd = op.forward(x, w, b)
        _, dw, db = op.backward(dy, x, w, b, mean, rstd)
        hat = ((x.double() - mean.double().repeat_interleave(c // groups, 1)[:, None])
               * rstd.double().repeat_interleave(c // groups, 1)[:, None])
        assert torch.all(db == 3.0)
        most = 2.0**-20 * (1 + hat[0, 0].abs() + hat[-1, 0].abs())
        assert ((dw.double() - hat[0, 0] - 2 * hat[-1, 0]).abs() <= most).all()
