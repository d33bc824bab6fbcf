"""Layer calls whose outputs are their inputs, through the C names: every one
gives what it gives with outputs of its own, bit for bit."""

import ctypes

import pytest

from tests import _gpu
from tests._gpu import torch

pytestmark = pytest.mark.gpu

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"f16": 0, "bf16": 1, "f32": 2}
ACT = {"none": 0, "silu": 1, "gelu": 2}


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


def draw(seed, *shape, dtype="f32", scale=1.0, offset=0.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale + offset).to(TORCH[dtype])


def same(a, b):
    return a.shape == b.shape and torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def stream():
    return torch.cuda.current_stream().cuda_stream


def norm_backward(tsx, op, dy, x, w, b, mean, rstd, dx, dw, db):
    """tsx_group_norm_backward with the caller's outputs."""
    need = ctypes.c_size_t()
    assert tsx.tsx_group_norm_workspace(ctypes.byref(op._desc), 1, 0, ctypes.byref(need)) == tsx.TSX_OK
    scratch = torch.empty(need.value, dtype=torch.uint8, device="cuda")
    p = [t.data_ptr() for t in (w, b, mean, rstd, dx, dw, db, scratch)]
    rc = tsx.tsx_group_norm_backward(ctypes.byref(op._desc), dy.data_ptr(), x.data_ptr(), None, None, *p,
                                     need.value, stream())
    assert rc == tsx.TSX_OK, tsx.tsx_last_error()


# rows read twice: several runs of channels and more CTAs than run at once; one run; then samples on chip, and tokens
@pytest.mark.parametrize("n,l,c,groups", [(8192, 1, 4096, 1), (3, 4000, 2048, 1), (2, 5000, 64, 4), (40, 30, 64, 8),
                                          (300, 1, 512, 8)])
def test_parameter_gradients_in_the_place_of_the_parameters(tsx, n, l, c, groups):
    op = tsx.GroupNorm("bf16", n, l, c, groups, act="silu")
    x, dy = draw(1, n, l, c, dtype="bf16"), draw(2, n, l, c, dtype="bf16")
    w, b = draw(3, c, scale=0.3, offset=1), draw(4, c, scale=0.3)
    _, mean, rstd = op.forward(x, w, b)
    want = op.backward(dy, x, w, b, mean, rstd)
    for cross in (False, True):
        dx, w2, b2 = torch.empty_like(x), w.clone(), b.clone()
        dw, db = (b2, w2) if cross else (w2, b2)
        norm_backward(tsx, op, dy, x, w2, b2, mean, rstd, dx, dw, db)
        for got, t in zip((dx, dw, db), want):
            assert same(got, t)
