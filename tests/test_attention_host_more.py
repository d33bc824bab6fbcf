"""More of the operators around attention on the host (no GPU): scales that are
refused, and angles of far positions."""

import ctypes
from fractions import Fraction

import numpy as np
import pytest

from tests.test_attention_host import A, batch, cache, heads, refused, tsx  # noqa: F401


def test_scales_that_are_refused(tsx, refused):  # noqa: F811
    """Those whose quotient by ln 2 is no fp32 number; their largest is taken (and
    the call refused for its workspace)."""
    def call(scale):
        return tsx.tsx_paged_attention(cache(tsx), batch(tsx), 4, 8, 1, scale, heads(tsx, A), heads(tsx, A), None, A, 0,
                                       None)

    for scale in (float("inf"), float("-inf"), float("nan"), 1.5 * 2.0**127, -2.0**128):
        refused(call(scale), tsx.TSX_ERR_INVALID, "scale")
        with pytest.raises(tsx.TsxError, match="scale"):
            tsx.PagedAttention("bf16", 4, 2, 64, 16, scale=scale)
    for scale in (2.0**127, -2.0**127, 0.0, 2.0**-149):
        refused(call(scale), tsx.TSX_ERR_INVALID, "workspace")
        tsx.PagedAttention("bf16", 4, 2, 64, 16, scale=scale)


def test_angles_of_far_positions(tsx):  # noqa: F811
    """A position times a frequency's turns, modulo 2^64, is the angle to |position|
    2^-63 of a turn (and the double-double quotient's 2^-98 of the frequency),
    whatever the position."""
    rng = np.random.default_rng(1)
    f = tsx.Rotary("f32", 1, 1, 128)
    values = list(f.frequencies) + [2.0**30, -(2.0**30), 123.456, -0.25]
    table, out = (ctypes.c_double * len(values))(*values), (ctypes.c_uint64 * len(values))()
    assert tsx.tsx_rotary_turns(len(values), table, out) == tsx.TSX_OK
    tau = Fraction("6.28318530717958647692528676655900576839433879875021164194988918461563281257241799725606965")
    far = [0, 1, -1, 2**31, -(2**31), 2**40, -(2**50), 2**62, -(2**63)] + [int(p) for p in rng.integers(-2**63, 2**63 - 1, 20)]
    for v, turns in zip(values, out):
        for p in far:
            off = (Fraction(p * turns % 2**64, 2**64) - Fraction(v) / tau * p) % 1
            assert min(off, 1 - off) <= abs(p) * (Fraction(1, 2**63) + abs(Fraction(v)) / tau / 2**98), (v, p)
