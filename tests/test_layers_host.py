"""The layer operators' host side (no GPU): argument checks of the C calls,
scratch sizes, and the plain definitions against themselves."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

from oracle import layers as ref


@pytest.fixture(scope="module")
def tsx():
    import __graft_entry__

    __graft_entry__.build()
    import pipelined_elementwise_streaming_gb300 as m

    return m


def desc(tsx, **kw):
    d = dict(dtype=1, param_dtype=2, act=1, groups=8, form=0, block=128, n=2, l=16, c=64, x_pitch=64, y_pitch=64,
             eps=1e-5)
    d.update(kw)
    return tsx.tsx_norm_desc(*d.values())


def workspace(tsx, backward=0, **kw):
    size = ctypes.c_size_t(99)
    rc = tsx.tsx_group_norm_workspace(ctypes.byref(desc(tsx, **kw)), backward, 0, ctypes.byref(size))
    if rc == tsx.TSX_OK:   # never more for aligned tensors
        least = ctypes.c_size_t(99)
        assert tsx.tsx_group_norm_workspace(ctypes.byref(desc(tsx, **kw)), backward, 1, ctypes.byref(least)) == rc
        assert least.value <= size.value
    return rc, size.value


def test_shapes_that_are_refused(tsx):
    for bad in (dict(dtype=3), dict(param_dtype=0), dict(act=3), dict(groups=0), dict(groups=7), dict(form=2),
                dict(block=16), dict(n=-1), dict(l=-1), dict(c=-8), dict(x_pitch=63), dict(y_pitch=0),
                dict(eps=-1e-5), dict(eps=float("nan")), dict(eps=float("inf")), dict(n=1 << 16, l=1 << 16)):
        rc, _ = workspace(tsx, **bad)
        assert rc == tsx.TSX_ERR_INVALID, bad
        assert tsx.tsx_last_error()
    assert tsx.tsx_group_norm_workspace(None, 0, 0, None) == tsx.TSX_ERR_INVALID
    head = (1, 4, 64, 64, 0, 128)
    for k, v in ((0, 9), (1, -1), (2, 1 << 31), (3, 63), (4, 5), (5, 100)):
        args = list(head)
        args[k] = v
        assert tsx.tsx_pack(*args, None, None, None, None) == tsx.TSX_ERR_INVALID, k
        assert tsx.tsx_unpack(*args, None, None, None, None) == tsx.TSX_ERR_INVALID, k
    assert tsx.tsx_pack(*head, None, None, None, None) == tsx.TSX_ERR_INVALID
    glu = (1, 4, 64, 64, 64, 1, 0, 128)
    assert tsx.tsx_gated_act(*glu, 16, 16, 16, 16, None, None, None, None) == tsx.TSX_ERR_INVALID
    assert "checkpoints" in tsx.tsx_last_error()
    assert tsx.tsx_gated_act_backward(*glu, 16, 16, None, 16, 16, None, None, 16, 16, None, None) == \
        tsx.TSX_ERR_INVALID


def test_empty_shapes_do_nothing(tsx):
    for rows, cols in ((0, 64), (4, 0)):
        assert tsx.tsx_pack(1, rows, cols, 64, 0, 128, None, None, None, None) == tsx.TSX_OK
        assert tsx.tsx_unpack(1, rows, cols, 64, 0, 128, None, None, None, None) == tsx.TSX_OK
        glu = (1, rows, cols, 64, 64, 1, 0, 128)
        assert tsx.tsx_gated_act(*glu, None, None, None, None, None, None, None, None) == tsx.TSX_OK
    assert workspace(tsx, n=0) == (tsx.TSX_OK, 0) and workspace(tsx, l=0) == (tsx.TSX_OK, 0)
    d = desc(tsx, n=0)
    assert tsx.tsx_group_norm(ctypes.byref(d), *[None] * 9, 0, None) == tsx.TSX_OK


@pytest.mark.parametrize("n,l,c,groups", [(1, 1, 64, 4), (8192, 1, 4096, 32), (1, 262144, 128, 32), (4, 100, 198, 11),
                                          (2, 3, 100000, 1), (1, 1, 1, 1), (1, 1 << 30, 1, 1), (1 << 30, 1, 1, 1)])
def test_scratch_is_small(tsx, n, l, c, groups):
    """A fraction of the tensor, or of a megabyte."""
    kw = dict(n=n, l=l, c=c, groups=groups, x_pitch=c, y_pitch=c)
    (rc, fwd), (rc2, bwd) = workspace(tsx, 0, **kw), workspace(tsx, 1, **kw)
    assert rc == rc2 == tsx.TSX_OK
    assert fwd <= bwd <= 64 * n * l * c + (64 << 20)


def test_definition_of_the_gradients():
    """The 64-bit gradients against central differences of the 64-bit forward
    pass: the error is of order h^2 = 1e-12 and 1e-16 / h."""
    rng = np.random.default_rng(1)
    n, l, c, groups, eps = 2, 5, 12, 3, 1e-3
    x, dy = rng.standard_normal((n, l, c)), rng.standard_normal((n, l, c))
    w, b = rng.standard_normal(c), rng.standard_normal(c)
    for kind in ("none", "silu", "gelu"):
        _, mean, rstd = ref.norm(x, w, b, groups, kind, eps)
        grads = ref.norm_backward(dy, x, w, b, mean, rstd, groups, kind)
        for k, at in enumerate((x, w, b)):
            v = rng.standard_normal(at.shape)

            def loss(t):
                args = [x, w, b]
                args[k] = at + t * v
                return (dy * ref.norm(*args, groups, kind, eps)[0]).sum()

            assert abs((loss(1e-6) - loss(-1e-6)) / 2e-6 - (grads[k] * v).sum()) < 1e-6


def test_definition_of_the_checkpoint():
    assert np.array_equal(ref.e4m3([0, 1, 1.0625, 1.1875, 448, 464, -447, 2.0**-9, 2.0**-10, 3 * 2.0**-10]),
                          [0, 1, 1, 1.25, 448, 448, -448, 2.0**-9, 0, 2.0**-8])
    x = np.array([[1.0, -127.0, 63.5, 0.5]], np.float32)
    q, scale = ref.hold(x, "int8", 32)
    assert scale[0, 0] == np.float32(127) * np.float32(1 / 127)
    assert np.array_equal(q[0, :2], [1, -127])


def test_header_is_plain_c(tmp_path):
    source = tmp_path / "client.c"
    source.write_text('#include "tsx_layers.h"\nint main(void) { return (int)sizeof(tsx_norm_desc) & 1; }\n')
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-pedantic", "-fsyntax-only", "-I", include, str(source)],
                   check=True)
