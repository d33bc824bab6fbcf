"""Plain definitions of the layer operators in numpy, 64 bits throughout:
group norm with an activation, gated activation, 8-bit checkpoints.

``hold`` alone follows fp32 steps, since the checkpoint's numbers are defined
by them (the scale is amax * fl(1 / top), the numbers x * fl(1 / scale) rounded
to nearest even); everything else is the formula.
"""

from __future__ import annotations

import numpy as np

TOP = {"int8": 127.0, "e4m3": 448.0}


def act(z, kind):
    """(act(z), act'(z))"""
    if kind == "none":
        return z, np.ones_like(z)
    if kind == "silu":
        p = 1 / (1 + np.exp(-z))
        return z * p, p * (1 + z * (1 - p))
    k = np.sqrt(2 / np.pi)
    t = np.tanh(k * (z + 0.044715 * z**3))
    return z / 2 * (1 + t), (1 + t) / 2 + z / 2 * (1 - t * t) * k * (1 + 3 * 0.044715 * z**2)


def norm(x, weight, bias, groups, kind, eps):
    """x [n, l, c] -> (y, mean [n, groups], rstd [n, groups])"""
    n, l, c = x.shape
    v = x.reshape(n, l, groups, c // groups)
    mean = v.mean((1, 3))
    var = ((v - mean[:, None, :, None]) ** 2).mean((1, 3))
    rstd = 1 / np.sqrt(var + eps)
    hat = ((v - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(n, l, c)
    return act(hat * weight + bias, kind)[0], mean, rstd


def norm_backward(dy, x, weight, bias, mean, rstd, groups, kind):
    """(dx, dweight, dbias) of sum(dy * y)"""
    n, l, c = x.shape
    per = c // groups
    m, r = (np.repeat(s, per, 1)[:, None, :] for s in (mean, rstd))
    hat = (x - m) * r
    dz = dy * act(hat * weight + bias, kind)[1]
    d = dz * weight

    def over_group(v):
        return np.repeat(v.reshape(n, l, groups, per).mean((1, 3)), per, 1)[:, None, :]

    return r * (d - over_group(d) - hat * over_group(d * hat)), (dz * hat).sum((0, 1)), dz.sum((0, 1))


def gated(gate, up, kind):
    return act(gate, kind)[0] * up


def gated_backward(dh, gate, up, kind):
    value, slope = act(gate, kind)
    return dh * up * slope, dh * value


def e4m3(v):
    """v rounded to the nearest e4m3 number, ties to even."""
    v = np.asarray(v, np.float64)
    unit = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0**-6))) - 3)
    return np.clip(np.rint(v / unit) * unit, -448, 448)


def hold(x, form, block):
    """fp32 x [rows, cols] -> (numbers as fp64, fp32 scales)"""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    q = np.zeros((rows, cols))
    scales = np.zeros((rows, -(-cols // block)), np.float32)
    for k in range(scales.shape[1]):
        b = x[:, k * block:(k + 1) * block]
        amax = np.abs(b).max(1)   # NaN stays NaN
        with np.errstate(all="ignore"):
            scale = amax * np.float32(1 / TOP[form])
            inv = np.float32(1) / scale
            tiny, bad = amax < np.float32(2.0**-119), ~np.isfinite(amax)
            v = np.where((tiny | bad)[:, None], 0, b * inv[:, None]).astype(np.float32)
        scales[:, k] = np.where(tiny, 0, np.where(bad, np.nan, scale))
        q[:, k * block:(k + 1) * block] = np.rint(v) if form == "int8" else e4m3(v)
    return q, scales


def stands_for(q, scales, block):
    with np.errstate(invalid="ignore"):
        return q * np.repeat(scales.astype(np.float64), block, 1)[:, : q.shape[1]]
