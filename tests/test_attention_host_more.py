"""More of the operators around attention on the host (no GPU): scales that are
refused."""

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
