"""Plain definitions of the operators around attention in numpy, 64 bits
throughout: rotary positions, norms of heads, appending to a paged cache,
attention over it."""

from __future__ import annotations

import numpy as np


def frequencies(rot, base=10000.0, scaling=None):
    """(radians to a position of each pair, amplitude)"""
    kind, *numbers = (None,) if scaling is None else scaling
    out, amplitude = [], 1.0
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if kind == "linear":
            f = f / numbers[0]
        elif kind == "ntk" and rot > 2:
            f = (base * numbers[0] ** (rot / (rot - 2))) ** (-2 * i / rot)
        elif kind == "yarn":
            factor, length, fast, slow = [*numbers, 32.0, 1.0][:4]

            def pair(turns):
                return rot * np.log(length / (2 * np.pi * turns)) / (2 * np.log(base))

            first, last = max(np.floor(pair(fast)), 0), min(np.ceil(pair(slow)), rot - 1)
            ramp = min(max((i - first) / max(last - first, 1e-3), 0), 1)
            f = f * (1 - ramp) + f / factor * ramp
            amplitude = 0.1 * np.log(factor) + 1
        out.append(f)
    return np.array(out), amplitude


def pairs(rot, layout):
    """Channels of the pairs' first and second members."""
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)


def turn(x, positions, freq, amplitude, layout, back=False):
    """x [tokens, heads, dim] with its first 2 len(freq) channels turned."""
    angle = np.asarray(positions, np.float64)[:, None] * freq
    c, s = amplitude * np.cos(angle)[:, None], amplitude * np.sin(angle)[:, None] * (-1 if back else 1)
    first, second = pairs(2 * len(freq), layout)
    out = x.copy()
    a, b = x[..., first], x[..., second]
    out[..., first], out[..., second] = a * c - b * s, a * s + b * c
    return out


def norm(x, weight, eps):
    """(x rstd weight, x rstd, rstd)"""
    rstd = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * rstd * weight, x * rstd, rstd


def norm_backward(d, x, weight, eps):
    """(dx, dweight) of sum(d * norm(x))"""
    _, hat, rstd = norm(x, weight, eps)
    g = d * weight
    return rstd * (g - hat * (g * hat).mean(-1, keepdims=True)), (d * hat).sum((0, 1))


def places(starts, lengths, pages, page_size, cache_pages, token):
    """(sequence, position, page or None) of a token, None for one of no
    sequence."""
    seqs = len(lengths)
    if not starts[0] <= token < starts[seqs]:
        return None
    b = int(np.searchsorted(starts, token, side="right")) - 1
    length = min(lengths[b], pages.shape[1] * page_size)
    p = length - starts[b + 1] + token
    if p < 0:
        return b, p, None
    page = pages[b, p // page_size]
    return b, p, int(page) if 0 <= page < cache_pages else None


def attend(q, k, v, starts, lengths, pages, scale):
    """(out, lse) of q [tokens, q_heads, dim] over caches [pages, page_size,
    heads, dim]; rows of no sequence are NaN.  Keys on pages that do not exist
    are passed over."""
    cache_pages, page_size, heads, dim = k.shape
    group = q.shape[1] // heads
    out, lse = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
    for t in range(len(q)):
        at = places(starts, lengths, pages, page_size, cache_pages, t)
        if at is None:
            continue
        b, p, _ = at
        out[t], lse[t] = 0, -np.inf
        seen = np.arange(p + 1)
        page = pages[b, seen // page_size] if p >= 0 else np.zeros(0, int)
        seen = seen[(page >= 0) & (page < cache_pages)]
        if not len(seen):
            continue
        page, slot = pages[b, seen // page_size], seen % page_size
        for h in range(heads):
            mine = slice(h * group, (h + 1) * group)
            x = q[t, mine] @ k[page, slot, h].T * scale
            top = x.max(-1, keepdims=True)
            w = np.exp(x - top)
            out[t, mine] = w @ v[page, slot, h] / w.sum(-1, keepdims=True)
            lse[t, mine] = top[:, 0] + np.log(w.sum(-1))
    return out, lse
