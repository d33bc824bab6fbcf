"""What the Python classes of the layer operators check before any GPU call."""

import types

import pytest


@pytest.fixture(scope="module")
def tsx():
    import __graft_entry__

    __graft_entry__.build()
    import pipelined_elementwise_streaming_gb300 as m

    return m


class Fake:
    """A tensor on a device that no test has."""

    def __init__(self, device):
        import torch

        self.device, self.is_cuda = torch.device("cuda", device), True

    def get_device(self):
        return self.device.index


def test_a_stream_of_another_device_is_refused(tsx, monkeypatch):
    """Not left aside for the current stream of the tensors' device."""
    import torch

    stream = types.SimpleNamespace(device=torch.device("cuda", 1), device_index=1)
    x = Fake(0)
    norm, glu, pack = tsx.GroupNorm("bf16", 2, 3, 8, 2), tsx.GatedAct("bf16", 4, 8), tsx.Packer("bf16", 4, 8)
    for op in (norm, glu, pack):
        monkeypatch.setattr(op, "_device", lambda: 0)
    for call in (lambda: norm.forward(x, x, x, stream=stream), lambda: norm.backward(x, x, x, x, x, x, stream=stream),
                 lambda: glu.forward(x, x, stream=stream), lambda: glu.backward(x, x, x, stream=stream),
                 lambda: pack.pack(x, stream=stream), lambda: pack.unpack((x, x), stream=stream)):
        with pytest.raises(tsx.TsxError) as e:
            call()
        assert e.value.code == tsx.TSX_ERR_INVALID and "stream" in str(e.value) and "cuda:1" in str(e.value)


def scratch(tsx, backward, n, l, c, groups, dtype=1, aligned=0):
    import ctypes

    d = tsx.tsx_norm_desc(dtype, 2, 1, groups, 0, 128, n, l, c, c, c, 1e-5)
    size = ctypes.c_size_t()
    assert tsx.tsx_group_norm_workspace(ctypes.byref(d), backward, aligned, ctypes.byref(size)) == tsx.TSX_OK
    return size.value


@pytest.mark.parametrize("n,l,c,groups", [
    (8192, 1, 4096, 1), (8192, 1, 4096, 8), (65536, 1, 4096, 1), (8192, 1, 2560, 32), (8192, 1, 1024, 1),
    (8192, 2, 4096, 8), (7088, 3, 352, 11), (7088, 3, 363, 11), (2000, 64, 256, 32), (2000, 1, 6000, 1),
    (300, 1, 65536, 1), (300, 2, 65536, 2), (16384, 1, 8192, 1), (16384, 1, 8191, 1), (1 << 20, 1, 33, 3),
    (1 << 20, 1, 40, 5), (1, 262144, 128, 32), (4, 16384, 512, 32), (256, 256, 512, 32), (100000, 7, 96, 32)])
@pytest.mark.parametrize("dtype,size", [(0, 2), (1, 2), (2, 4)])
def test_scratch_of_the_gradient_does_not_grow_with_the_samples(tsx, n, l, c, groups, dtype, size):
    """Sums for dweight and dbias: 16 MB, or one slice of two floats to a
    channel; beside them a few bytes to a sample's group and range."""
    slices = max(16 << 20, 8 * c)
    pieces = -(-c // groups // 2048)
    parts = 8 * groups * (n + 608) * pieces + 16
    for backward in (0, 1):
        for aligned in (0, 1):
            assert scratch(tsx, backward, n, l, c, groups, dtype, aligned) <= parts + backward * slices
    assert scratch(tsx, 1, n, l, c, groups, dtype) <= n * l * c * size // 2 + (18 << 20)


# ------------------------------------------------------------- refusals
# Calls that are refused look at no memory and launch nothing, so numbers stand for addresses here.

A = 1 << 20          # aligned to anything
SIZES = (1, 4, 64)   # bf16, rows, cols


@pytest.fixture
def refused(tsx):
    import torch

    if torch.cuda.is_available():
        pytest.skip("stands-in for addresses stay off GPUs")

    def check(rc, code, word):
        assert rc == code and word in tsx.tsx_last_error()

    return check


def test_constructors(tsx):
    for make in (lambda: tsx.Packer("f64", 4, 64), lambda: tsx.Packer("bf16", 4, 64, block=48),
                 lambda: tsx.Packer("bf16", 4, 64, form="int4"), lambda: tsx.GatedAct("bf16", 4, 64, act="relu"),
                 lambda: tsx.GatedAct("i8", 4, 64), lambda: tsx.GatedAct("bf16", 4, 64, form="e5m2"),
                 lambda: tsx.GatedAct("bf16", 4, 64, block=0), lambda: tsx.GroupNorm("bf16", 1, 4, 64, 7),
                 lambda: tsx.GroupNorm("bf16", 1, 4, 64, 0), lambda: tsx.GroupNorm("bf16", 1, 4, 64, -8),
                 lambda: tsx.GroupNorm("bf16", 1, 4, 64, 8, eps=-1.0),
                 lambda: tsx.GroupNorm("bf16", 1, 4, 64, 8, eps=float("nan")),
                 lambda: tsx.GroupNorm("bf16", 1, 4, 64, 8, act="tanh"),
                 lambda: tsx.GroupNorm("bf16", 1, 4, 64, 8, param_dtype="f16"),
                 lambda: tsx.GroupNorm("bf16", 1, 4, 64, 8, param_dtype="f64"),
                 lambda: tsx.GroupNorm("bf16", 1, 4, 64, 8, x_pitch=63),
                 lambda: tsx.GroupNorm("bf16", 1, 4, 64, 8, y_pitch=8),
                 lambda: tsx.GroupNorm("bf16", -1, 4, 64, 8), lambda: tsx.GroupNorm("bf16", 1, 4, -64, 8),
                 lambda: tsx.GroupNorm("bf16", 1 << 20, 1 << 20, 64, 8)):
        with pytest.raises(tsx.TsxError) as e:
            make()
        assert e.value.code == tsx.TSX_ERR_INVALID and len(str(e.value)) > 15


def test_packing(tsx, refused):
    for call in (tsx.tsx_pack, tsx.tsx_unpack):
        head = (*SIZES, 64, 0, 128)
        for k in range(3):
            args = [A, A, A]
            args[k] = None
            refused(call(*head, *args, None), tsx.TSX_ERR_INVALID, "required")
        # the tensor and the scales; bytes may lie anywhere
        x, scale = (0, 2) if call is tsx.tsx_pack else (2, 1)
        for k, off in ((x, 1), (scale, 2)):
            args = [A, A, A]
            args[k] += off
            refused(call(*head, *args, None), tsx.TSX_ERR_ALIGN, "aligned")
        refused(call(1, 4, 1 << 30, 1 << 30, 0, 128, A, A, A, None), tsx.TSX_ERR_UNSUPPORTED, "too long")
        refused(call(1, (1 << 31) - 1, 64, 64, 0, 128, A, A, A, None), tsx.TSX_ERR_INVALID, "2^31")


def test_gated(tsx, refused):
    head = (*SIZES, 64, 64, 1, 0, 128)
    for k, v, word in ((0, 3, "dtype"), (1, -1, "rows"), (2, 1 << 31, "cols"), (3, 63, "pitch"), (4, 63, "pitch"),
                       (5, 3, "activation"), (5, -1, "activation"), (6, 2, "form"), (7, 16, "block")):
        args = list(head)
        args[k] = v
        refused(tsx.tsx_gated_act(*args, A, A, A, *[None] * 4, None), tsx.TSX_ERR_INVALID, word)
        refused(tsx.tsx_gated_act_backward(*args, A, A, A, *[None] * 4, A, A, None, None), tsx.TSX_ERR_INVALID, word)
    for k in range(3):
        args = [A, A, A]
        args[k] = None
        refused(tsx.tsx_gated_act(*head, *args, *[None] * 4, None), tsx.TSX_ERR_INVALID, "required")
        args[k] = A + 1
        refused(tsx.tsx_gated_act(*head, *args, *[None] * 4, None), tsx.TSX_ERR_ALIGN, "aligned")
    for k in range(4):   # three of the four
        held = [A] * 4
        held[k] = None
        refused(tsx.tsx_gated_act(*head, A, A, A, *held, None), tsx.TSX_ERR_INVALID, "checkpoints")
        refused(tsx.tsx_gated_act_backward(*head, A, None, None, *held, A, A, None, None), tsx.TSX_ERR_INVALID,
                "checkpoints")
    for k in (1, 3):
        held = [A] * 4
        held[k] += 2
        refused(tsx.tsx_gated_act(*head, A, A, A, *held, None), tsx.TSX_ERR_ALIGN, "aligned")
        refused(tsx.tsx_gated_act_backward(*head, A, None, None, *held, A, A, None, None), tsx.TSX_ERR_ALIGN,
                "aligned")
    refused(tsx.tsx_gated_act_backward(*head, A, A, A, A, A, A, A, A, A, None, None), tsx.TSX_ERR_INVALID,
            "checkpoints")
    for k in (0, 7, 8):
        args = [A, A, A, *[None] * 4, A, A, None]
        args[k] = None
        refused(tsx.tsx_gated_act_backward(*head, *args, None), tsx.TSX_ERR_INVALID, "required")
    for k in (0, 1, 2, 7, 8, 9):
        args = [A, A, A, *[None] * 4, A, A, None]
        args[k] = A + 1
        refused(tsx.tsx_gated_act_backward(*head, *args, None), tsx.TSX_ERR_ALIGN, "aligned")
    long = (1, 4, 1 << 30, 1 << 30, 1 << 30, 1, 0, 128)
    refused(tsx.tsx_gated_act(*long, A, A, A, *[None] * 4, None), tsx.TSX_ERR_UNSUPPORTED, "too long")
    refused(tsx.tsx_gated_act_backward(*long, A, A, A, *[None] * 4, A, A, None, None), tsx.TSX_ERR_UNSUPPORTED,
            "too long")


def test_norm(tsx, refused):
    import ctypes

    def desc(dtype=1, param=2, act=0, groups=8, n=2, l=300, c=64, pitch=None):
        return ctypes.byref(tsx.tsx_norm_desc(dtype, param, act, groups, 0, 128, n, l, c, pitch or c, pitch or c, 1e-5))

    def forward(d=None, x=A, w=A, b=A, y=A, mean=A, rstd=A, q=None, scale=None, work=A, size=1 << 30):
        return tsx.tsx_group_norm(d or desc(), x, w, b, y, mean, rstd, q, scale, work, size, None)

    def backward(d=None, dy=A, x=A, q=None, scale=None, w=A, b=A, mean=A, rstd=A, dx=A, dw=A, db=A, work=A,
                 size=1 << 30):
        return tsx.tsx_group_norm_backward(d or desc(), dy, x, q, scale, w, b, mean, rstd, dx, dw, db, work, size,
                                           None)

    invalid, align = tsx.TSX_ERR_INVALID, tsx.TSX_ERR_ALIGN
    refused(tsx.tsx_group_norm(None, *[A] * 9, 0, None), invalid, "descriptor")
    for call in (forward, backward):
        refused(call(desc(param=0)), invalid, "fp32 or of the element type")
        refused(call(desc(act=7)), invalid, "activation")
        refused(call(desc(groups=5)), invalid, "groups")
        refused(call(desc(pitch=63)), invalid, "pitch")
        refused(call(desc(c=1 << 30, groups=1, l=1)), tsx.TSX_ERR_UNSUPPORTED, "too long")
    for name in ("x", "w", "b", "y", "mean", "rstd"):
        refused(forward(**{name: None}), invalid, "required")
        refused(forward(**{name: A + 1}), align, "aligned")
    for name in ("dy", "w", "b", "mean", "rstd", "dx", "dw", "db"):
        refused(backward(**{name: None}), invalid, "required")
        refused(backward(**{name: A + 1}), align, "aligned")
    refused(forward(desc(param=1), w=A + 1), align, "aligned")
    refused(forward(q=A), invalid, "together")
    refused(forward(scale=A), invalid, "together")
    refused(forward(q=A + 1, scale=A + 2), align, "aligned")
    for kw in (dict(x=None), dict(q=A, scale=A), dict(x=None, q=A), dict(x=None, scale=A)):
        refused(backward(**kw), invalid, "checkpoint")
    refused(backward(x=None, q=A, scale=A + 2), align, "aligned")
    refused(backward(x=A + 1), align, "aligned")
    # scratch: rows read twice need it in both passes
    rows = dict(d=desc(l=9000, groups=4))
    for call in (forward, backward):
        refused(call(**rows, work=None), invalid, "workspace")
        refused(call(**rows, work=A + 8), align, "workspace")
        need = scratch(tsx, call is backward, 2, 9000, 64, 4, aligned=1)
        assert need > 0
        refused(call(**rows, size=need - 1), invalid, "workspace")
    refused(backward(work=None), invalid, "workspace")
    # tensors without elements need nothing but what is written
    assert forward(desc(n=0), *[None] * 6, work=None, size=0) == tsx.TSX_OK
    assert forward(desc(c=0, pitch=8), *[None] * 6, work=None, size=0) == tsx.TSX_OK
    refused(forward(desc(l=0), *[None] * 6), invalid, "mean")
    refused(backward(desc(l=0), dw=None), invalid, "dweight")
