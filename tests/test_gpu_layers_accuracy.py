"""fp32 activations and slopes, one argument at a time, within the errors that
the header states, against 64 bits.

U = 2^-24 is fp32's rounding.  The sigmoid p of u (u = z for silu, 2 k (z +
0.044715 z^3) for gelu) carries, relative to p, D = 2^-21 (1 + |u| (1 - p)): 2
ulps of the exponential (2^-22), 1 of the reciprocal (2^-23), the sum's rounding
(U), and its argument's: -z log2(e) with the constant's and the product's, gelu's
with three roundings and two constants more, each U |u|, on 2^u's share 1 - p of
the denominator.
  value z p          : |z| p D, and U for the product
  slope p + z p (1 - p) w, w = 1 (silu) or 2 k (1 + 0.134145 z^2) (gelu)
                     : p D, |z| w p (1 - p) D, |z| w p (p D + U) for 1 - p, and
                       8 U for the products and the sum
and 2^-118 for what becomes 0.  gelu's argument is taken at |z| <= 24, where p
is 0 or 1 within those bounds."""

import numpy as np
import pytest

from tests import _gpu
from tests._gpu import torch

pytestmark = pytest.mark.gpu

U = 2.0**-24
K2 = 2 * np.sqrt(2 / np.pi)


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


def arguments():
    rng = np.random.default_rng(1)
    z = np.concatenate([np.linspace(-130, 130, 200001), np.linspace(-12, 12, 300001), rng.standard_normal(300000),
                        np.exp2(rng.uniform(-120, 6, 100000)) * rng.choice([-1, 1], 100000),
                        [0.0, -0.0, 87.3, -87.3, 88.8, -88.8, 24, -24, 1e4, -1e4]])
    return z.astype(np.float32)


def exact(z, act):
    """(value, slope, p, 1 - p, u, w) in 64 bits; 1 - p without cancellation"""
    u, w = (z, np.ones_like(z)) if act == "silu" else (K2 * (z + 0.044715 * z**3), K2 * (1 + 0.134145 * z**2))
    with np.errstate(over="ignore"):
        p, rest = 1 / (1 + np.exp(-u)), 1 / (1 + np.exp(u))
    return z * p, p + z * p * rest * w, p, rest, u, w


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_values_and_slopes(tsx, act):
    z32 = arguments()
    z = z32.astype(np.float64)
    value, slope, p, rest, u, w = exact(z, act)
    d = 2.0**-21 * (1 + np.abs(u) * rest)
    e_value = np.abs(z) * p * d * 1.001 + 2 * U * np.abs(value) + 2.0**-118
    zw = np.abs(z) * w * p
    e_slope = 1.001 * (p * d + zw * (rest * d + p * d + U)) + 8 * U * (p + zw * rest) + 2.0**-118
    gate = torch.from_numpy(z32).cuda()[None]
    one = torch.ones_like(gate)
    op = tsx.GatedAct("f32", 1, z.size, act=act)

    def near(got, want, bound, what):
        got = got[0].cpu().double().numpy()
        off = np.abs(got - want) - bound
        k = int(np.argmax(off))
        assert off[k] <= 0, f"{act} {what} at {z[k]!r}: {got[k]!r} for {want[k]!r}, bound {bound[k]:.3g}"

    near(op.forward(gate, one), value, e_value, "value")
    dgate, dup, h = op.backward(one, gate, one, recompute=True)
    near(dgate, slope, e_slope, "slope")
    near(dup, value, e_value, "value in the backward pass")
    near(h, value, e_value, "value again")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_the_norms_share_them(tsx, act):
    """A norm whose statistics leave its input as it is (one group of +-1 has
    mean 0 and, with eps 0, rstd 1) and a weight of 0: y = act(bias) and dbias =
    act'(bias), one argument to a channel."""
    z32 = arguments()
    z32 = z32[: z32.size // 64 * 64]
    z = z32.astype(np.float64)
    value, slope, p, rest, u, w = exact(z, act)
    d = 2.0**-21 * (1 + np.abs(u) * rest)
    c = z.size
    x = torch.ones(1, 2, c, device="cuda")
    x[:, 1] = -1
    dy = torch.zeros_like(x)
    dy[:, 0] = 1
    op = tsx.GroupNorm("f32", 1, 2, c, c // 64, act=act, eps=0.0)
    bias, weight = torch.from_numpy(z32).cuda(), torch.zeros(c, device="cuda")
    y, mean, rstd = op.forward(x, weight, bias)
    assert torch.all(mean == 0) and (rstd - 1).abs().max() <= 2.0**-22
    _, _, dbias = op.backward(dy, x, weight, bias, mean, rstd)
    zw = np.abs(z) * w * p
    e_value = np.abs(z) * p * d * 1.001 + 2 * U * np.abs(value) + 2.0**-118
    off = np.abs(y[0, 0].cpu().double().numpy() - value) - e_value
    assert off.max() <= 0, z[np.argmax(off)]
    # silu's slope comes from -z log2(e) and ln(2): one more rounding each
    off = np.abs(dbias.cpu().double().numpy() - slope) - (1.001 * (p * d + zw * (rest * d + p * d + 2 * U)) +
                                                          10 * U * (p + zw * rest) + 2.0**-118)
    assert off.max() <= 0, z[np.argmax(off)]
