"""What a layer call reports when a launch fails on the host, and that a later
call is not blamed for it."""

import ctypes

import pytest

from tests import _gpu
from tests._gpu import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


def test_a_failed_launch_is_reported_once(tsx):
    """While a stream that waits for the legacy one is captured, a launch on
    the legacy stream is refused by the runtime.  The call says so, and the
    next one, after the capture, is as good as ever."""
    cu = ctypes.CDLL("libcuda.so.1")
    n, l, c, groups = 2, 600, 64, 4
    x = torch.randn(n, l, c, device="cuda").bfloat16()
    w, b = torch.ones(c, device="cuda"), torch.zeros(c, device="cuda")
    op = tsx.GroupNorm("bf16", n, l, c, groups)
    pack = tsx.Packer("bf16", n * l, c)
    want, held = op.forward(x, w, b), pack.pack(x.view(n * l, c))
    q, scale = torch.empty_like(held.q), torch.empty_like(held.scale)
    y, mean, rstd = (torch.empty_like(t) for t in want)
    size = op._scratch[0][0]
    scratch = torch.empty(size + 16, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def norm(stream):
        return tsx.tsx_group_norm(ctypes.byref(op._desc), *(t.data_ptr() for t in (x, w, b, y, mean, rstd)), None, None,
                                  scratch.data_ptr(), size, stream)

    def packed(stream):
        return tsx.tsx_pack(*pack._head, x.data_ptr(), q.data_ptr(), scale.data_ptr(), stream)

    for first in (norm, packed):
        for then in (norm, packed):
            side, graph = ctypes.c_void_p(), ctypes.c_void_p()
            assert cu.cuStreamCreate(ctypes.byref(side), 0) == 0
            assert cu.cuStreamBeginCapture_v2(side, 0) == 0
            rc, message = first(None), tsx.tsx_last_error()
            cu.cuStreamEndCapture(side, ctypes.byref(graph))   # the refusal has ended the capture
            assert cu.cuStreamDestroy_v2(side) == 0
            assert rc == tsx.TSX_ERR_CUDA and message
            for t in (y, mean, rstd, scale):
                t.zero_()
            assert then(None) == tsx.TSX_OK, tsx.tsx_last_error()
            torch.cuda.synchronize()
            if then is norm:
                assert all(torch.equal(p, r) for p, r in zip((y, mean, rstd), want))
            else:
                assert torch.equal(q, held.q) and torch.equal(scale, held.scale)
