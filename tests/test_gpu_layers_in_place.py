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


# dtype, rows, cols, pitch: vectors; fp32 rows that start half a sector apart; single elements
GATED = [("bf16", 130, 4096, 4096), ("f16", 33, 200, 208), ("f32", 57, 1000, 1004), ("f32", 64, 256, 256),
         ("bf16", 41, 333, 333), ("f32", 37, 127, 130)]


@pytest.mark.parametrize("dtype,rows,cols,pitch", GATED)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated(tsx, dtype, rows, cols, pitch, act):
    def wide(seed, **kw):
        return draw(seed, rows, pitch, dtype=dtype, **kw)[:, :cols]

    def copy(t):
        u = torch.empty(rows, pitch, dtype=t.dtype, device="cuda")[:, :cols]
        return u.copy_(t)

    op = tsx.GatedAct(dtype, rows, cols, act=act, in_pitch=pitch, out_pitch=pitch)
    gate, up, dh = wide(1, scale=2), wide(2), wide(3)
    h, cg, cu = op.forward(gate, up, checkpoint=True)
    for held in (False, True):
        for k in range(2):   # h in the place of gate, then of up
            g, u = copy(gate), copy(up)
            got = op.forward(g, u, out=(g, u)[k], checkpoint=held)
            assert same(got[0] if held else got, h)
            assert same((u, g)[k], (up, gate)[k])
            if held:
                assert all(same(p, q) for p, q in zip((*got[1], *got[2]), (*cg, *cu)))
    head = (CODE[dtype], rows, cols, pitch, pitch, ACT[act], 0, 128)
    for src in ("tensors", "checkpoints"):
        if src == "tensors":
            dgate, dup, h = op.backward(dh, gate, up, recompute=True)
        else:
            dgate, dup, h = op.backward(dh, cg, cu, recompute=True)
        # (dgate, dup, h) in the places of (gate, up, dh), crosswise, and one of them in dh's
        for where in ("gud", "ugd", "d--", "-d-", "--d", "g-d", "-g-", "u--"):
            if src == "checkpoints" and ("g" in where or "u" in where):
                continue
            t = {"g": copy(gate), "u": copy(up), "d": copy(dh)}
            outs = [t[k] if k != "-" else torch.empty(rows, pitch, dtype=dh.dtype, device="cuda")[:, :cols]
                    for k in where]
            if src == "tensors":
                saved = (t["g"].data_ptr(), t["u"].data_ptr(), None, None, None, None)
            else:
                saved = (None, None, *(p.data_ptr() for p in (*cg, *cu)))
            rc = tsx.tsx_gated_act_backward(*head, t["d"].data_ptr(), *saved, *(o.data_ptr() for o in outs), stream())
            assert rc == tsx.TSX_OK, tsx.tsx_last_error()
            for got, want in zip(outs, (dgate, dup, h)):
                assert same(got, want), (src, where)


# n, l, c, groups, pitch: tokens; samples on chip; rows read twice, in ranges, in clusters and groups wider than a
# CTA's row (whose checkpoint is packed first); odd channels; rows that start half a sector apart
NORMS = [(300, 1, 512, 8, 512), (300, 1, 512, 8, 516), (40, 30, 64, 8, 68), (2, 1000, 320, 32, 324),
         (2, 9000, 64, 4, 68), (1, 60000, 64, 4, 64), (2, 3, 6000, 2, 6004), (9, 1, 5000, 1, 5000), (3, 50, 33, 3, 33),
         (2, 9000, 30, 5, 31)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,l,c,groups,pitch", NORMS)
def test_norm(tsx, dtype, n, l, c, groups, pitch):
    def wide(seed, **kw):
        return draw(seed, n, l, pitch, dtype=dtype, **kw)[..., :c]

    def copy(t):
        u = torch.empty(n, l, pitch, dtype=t.dtype, device="cuda")[..., :c]
        return u.copy_(t)

    op = tsx.GroupNorm(dtype, n, l, c, groups, act="silu", x_pitch=pitch, y_pitch=pitch)
    x, dy = wide(1, scale=1.5, offset=0.3), wide(2)
    w, b = draw(3, c, scale=0.3, offset=1), draw(4, c, scale=0.3)
    want = op.forward(x, w, b)
    t = copy(x)
    assert all(same(p, q) for p, q in zip(op.forward(t, w, b, out=t), want))
    y, mean, rstd, saved = op.forward(x, w, b, checkpoint=True)
    t = copy(x)
    got = op.forward(t, w, b, out=t, checkpoint=True)
    assert all(same(p, q) for p, q in zip((*got[:3], *got[3]), (y, mean, rstd, *saved)))
    want = op.backward(dy, x, w, b, mean, rstd)
    t = copy(x)
    assert all(same(p, q) for p, q in zip(op.backward(dy, t, w, b, mean, rstd, out=t), want))
    t = copy(dy)
    assert all(same(p, q) for p, q in zip(op.backward(t, x, w, b, mean, rstd, out=t), want))
    want = op.backward(dy, saved, w, b, mean, rstd)
    t = copy(dy)
    assert all(same(p, q) for p, q in zip(op.backward(t, saved, w, b, mean, rstd, out=t), want))
