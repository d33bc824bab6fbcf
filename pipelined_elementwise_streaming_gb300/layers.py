"""The layer operators of libtsx (include/tsx_layers.h) for torch tensors.

``GroupNorm``, ``GatedAct`` and ``Packer`` hold a shape and what the C calls
need of it; they own no device memory and may be used from several streams::

    norm = GroupNorm("bf16", n, l, c, groups=32, act="silu")
    y, mean, rstd, saved = norm.forward(x, weight, bias, checkpoint=True)
    dx, dweight, dbias = norm.backward(dy, saved, weight, bias, mean, rstd)

    glu = GatedAct("bf16", rows, cols, act="silu", in_pitch=2 * cols)
    h, gate8, up8 = glu.forward(both[:, :cols], both[:, cols:], checkpoint=True)
    dgate, dup = glu.backward(dh, gate8, up8)

Autograd does not see the calls: what they return has no graph, also for inputs
that require gradients.  examples/train_block.py wraps forward and backward in
autograd functions.

Results and scratch come from torch's allocator for the stream that the call
runs on; tensors that the caller passes with ``stream=`` belong to the caller,
who keeps them alive until that stream's work is done.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

from . import DTYPES, TSX_ERR_INVALID, TSX_OK, TsxError, lib, tsx_last_error

ACTS = {"none": 0, "silu": 1, "gelu": 2}
FORMS = {"int8": 0, "e4m3": 1}


class tsx_norm_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "param_dtype", "act", "groups", "form", "block")] + \
               [(n, ctypes.c_int64) for n in ("n", "l", "c", "x_pitch", "y_pitch")] + [("eps", ctypes.c_float)]


def _declare():
    p, i, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    sizes = [i, i64, i64, i64, i, i]
    lib.tsx_pack.argtypes = sizes + [p] * 4
    lib.tsx_unpack.argtypes = sizes + [p] * 4
    gated = [i, i64, i64, i64, i64, i, i, i]
    lib.tsx_gated_act.argtypes = gated + [p] * 8
    lib.tsx_gated_act_backward.argtypes = gated + [p] * 11
    d = ctypes.POINTER(tsx_norm_desc)
    lib.tsx_group_norm_workspace.argtypes = [d, i, i, ctypes.POINTER(ctypes.c_size_t)]
    lib.tsx_group_norm.argtypes = [d] + [p] * 9 + [ctypes.c_size_t, p]
    lib.tsx_group_norm_backward.argtypes = [d] + [p] * 12 + [ctypes.c_size_t, p]


_declare()

tsx_pack = lib.tsx_pack
tsx_unpack = lib.tsx_unpack
tsx_gated_act = lib.tsx_gated_act
tsx_gated_act_backward = lib.tsx_gated_act_backward
tsx_group_norm_workspace = lib.tsx_group_norm_workspace
tsx_group_norm = lib.tsx_group_norm
tsx_group_norm_backward = lib.tsx_group_norm_backward


class Checkpoint(NamedTuple):
    """A tensor held in 8 bits: q (int8 or float8_e4m3fn) stands for
    q * scale, one fp32 scale to a block of a row's channels.  The calls take
    any (q, scale) tuple."""
    q: object
    scale: object


def _call(rc: int) -> None:
    if rc != TSX_OK:
        raise TsxError(rc, tsx_last_error())


def _invalid(message: str):
    raise TsxError(TSX_ERR_INVALID, message)


def _named(table: dict, key, what: str) -> int:
    if key not in table:
        _invalid(f"unknown {what} {key!r}: one of {', '.join(map(str, table))}")
    return table[key]


class _Layer:
    """What the layers share: their torch types, the checks of tensors, and
    where results live.  Calls are short enough for their marshalling to show,
    so each tensor is first held against the exact strides of its layout, and
    only one that differs is looked at closely."""

    def __init__(self, dtype: str, rows: int, cols: int, form: str, block: int):
        import torch

        self._torch = torch
        self._dtype_code = _named(DTYPES, dtype, "dtype")
        self._form_code = _named(FORMS, form, "8-bit form")
        self.dtype, self.rows, self.cols, self.form, self.block = dtype, int(rows), int(cols), form, int(block)
        self._torch_dtype = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self._f32, self._byte = torch.float32, torch.uint8
        self._q_dtype = torch.int8 if form == "int8" else torch.float8_e4m3fn
        if self.block not in (32, 64, 128):
            _invalid("block must be 32, 64 or 128")
        self._q_shape, self._scale_shape = (self.rows, self.cols), (self.rows, -(-self.cols // self.block))
        self._shape = self._q_shape
        self._device = torch._C._cuda_getDevice
        self._stream = torch._C._cuda_getCurrentRawStream
        self._new = torch.empty

    def _strides_of(self, pitch: int):
        """Strides of the layer's shape with this row pitch."""
        strides = [1]
        for k in range(len(self._shape) - 2, -1, -1):
            strides.append(pitch if len(strides) == 1 else strides[-1] * self._shape[k + 1])
        return tuple(reversed(strides))

    def _ptr(self, t, strides, name: str, dev: int) -> int:
        """The address of t, a tensor of the layer's shape and type with these
        strides (those of dimensions of one element aside)."""
        if t.dtype is self._torch_dtype and t.shape == self._shape and t.stride() == strides and t.get_device() == dev:
            return t.data_ptr()
        if t.dtype is not self._torch_dtype or t.get_device() != dev:
            _invalid(f"{name} must be a {self.dtype} tensor on cuda:{dev}, got {t.dtype} on {t.device}")
        if tuple(t.shape) != self._shape:
            _invalid(f"{name} must have shape {list(self._shape)}, got {list(t.shape)}")
        if t.numel() and any(a != b and n != 1 for a, b, n in zip(t.stride(), strides, t.shape)):
            _invalid(f"{name} must have strides {list(strides)}, got {list(t.stride())}")
        return t.data_ptr()

    def _saved(self, c, name: str, dev: int):
        q, scale = c
        if (q.dtype is not self._q_dtype or scale.dtype is not self._f32 or q.get_device() != dev
                or scale.get_device() != dev):
            _invalid(f"{name} must be an {self.form} checkpoint with fp32 scales on cuda:{dev}")
        if (q.shape != self._q_shape or scale.shape != self._scale_shape or not q.is_contiguous()
                or not scale.is_contiguous()):
            _invalid(f"{name} must hold dense {list(self._q_shape)} numbers and {list(self._scale_shape)} scales")
        return q.data_ptr(), scale.data_ptr()

    def _vector(self, t, shape, dtype, name: str, dev: int) -> int:
        if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or (
                t.shape != shape and t.numel() != _count(shape)):
            _invalid(f"{name} must be {_count(shape)} contiguous {dtype} values on cuda:{dev}")
        return t.data_ptr()

    def _empty(self, device, pitch: int):
        if pitch == self.cols:
            return self._new(self._shape, dtype=self._torch_dtype, device=device)
        wide = self._new((*self._shape[:-1], pitch), dtype=self._torch_dtype, device=device)
        return wide.as_strided(self._shape, wide.stride())

    def _new_checkpoint(self, device) -> Checkpoint:
        return Checkpoint(self._new(self._q_shape, dtype=self._q_dtype, device=device),
                          self._new(self._scale_shape, dtype=self._f32, device=device))

    def _elsewhere(self, call, first, stream, args):
        """The call with the tensors' device and the stream made current."""
        t = self._torch
        if not first.is_cuda:
            _invalid("tensors must be on a CUDA device")
        if stream is not None and stream.device != first.device:
            _invalid(f"the stream is one of {stream.device}, the tensors are on {first.device}")
        with t.cuda.device(first.device), t.cuda.stream(stream):
            return call(self, *args)


def _count(shape) -> int:
    n = 1
    for k in shape:
        n *= k
    return n


class Packer(_Layer):
    """Tensors [rows, cols] to 8 bits and back (tsx_pack, tsx_unpack)."""

    def __init__(self, dtype: str, rows: int, cols: int, form: str = "int8", block: int = 128,
                 pitch: int | None = None):
        super().__init__(dtype, rows, cols, form, block)
        self.pitch = self.cols if pitch is None else int(pitch)
        self._strides = self._strides_of(self.pitch)
        self._head = (self._dtype_code, self.rows, self.cols, self.pitch, self._form_code, self.block)

    def pack(self, x, out: Checkpoint | None = None, stream=None) -> Checkpoint:
        dev = x.get_device()
        if stream is not None or dev != self._device():
            return self._elsewhere(Packer.pack, x, stream, (x, out))
        px = self._ptr(x, self._strides, "x", dev)
        if out is None:
            out = self._new_checkpoint(x.device)
            pq, ps = out.q.data_ptr(), out.scale.data_ptr()
        else:
            pq, ps = self._saved(out, "out", dev)
        rc = tsx_pack(*self._head, px, pq, ps, self._stream(dev))
        if rc:
            _call(rc)
        return out

    def unpack(self, saved: Checkpoint, out=None, stream=None):
        dev = saved[0].get_device()
        if stream is not None or dev != self._device():
            return self._elsewhere(Packer.unpack, saved[0], stream, (saved, out))
        pq, ps = self._saved(saved, "saved", dev)
        if out is None:
            out = self._empty(saved[0].device, self.pitch)
            po = out.data_ptr()
        else:
            po = self._ptr(out, self._strides, "out", dev)
        rc = tsx_unpack(*self._head, pq, ps, po, self._stream(dev))
        if rc:
            _call(rc)
        return out


class GatedAct(_Layer):
    """h = act(gate) * up over [rows, cols] (tsx_gated_act and its backward
    pass).  in_pitch: the row pitch of gate and up and of their gradients
    (2 * cols for the halves of one tensor: the gradients then are the halves
    of one new tensor too); out_pitch: of h and dh."""

    def __init__(self, dtype: str, rows: int, cols: int, act: str = "silu", form: str = "int8", block: int = 128,
                 in_pitch: int | None = None, out_pitch: int | None = None):
        super().__init__(dtype, rows, cols, form, block)
        self.act = act
        self.in_pitch = self.cols if in_pitch is None else int(in_pitch)
        self.out_pitch = self.cols if out_pitch is None else int(out_pitch)
        self._in, self._out = self._strides_of(self.in_pitch), self._strides_of(self.out_pitch)
        self._halves = self.in_pitch >= 2 * self.cols
        self._head = (self._dtype_code, self.rows, self.cols, self.in_pitch, self.out_pitch,
                      _named(ACTS, act, "activation"), self._form_code, self.block)

    def forward(self, gate, up, out=None, checkpoint: bool = False, stream=None):
        """h, or with checkpoint (h, gate's Checkpoint, up's Checkpoint)."""
        dev = gate.get_device()
        if stream is not None or dev != self._device():
            return self._elsewhere(GatedAct.forward, gate, stream, (gate, up, out, checkpoint))
        pg, pu = self._ptr(gate, self._in, "gate", dev), self._ptr(up, self._in, "up", dev)
        if out is None:
            out = self._empty(gate.device, self.out_pitch)
            ph = out.data_ptr()
        else:
            ph = self._ptr(out, self._out, "out", dev)
        if not checkpoint:
            rc = tsx_gated_act(*self._head, pg, pu, ph, None, None, None, None, self._stream(dev))
            if rc:
                _call(rc)
            return out
        cg, cu = self._new_checkpoint(gate.device), self._new_checkpoint(gate.device)
        rc = tsx_gated_act(*self._head, pg, pu, ph, cg.q.data_ptr(), cg.scale.data_ptr(), cu.q.data_ptr(),
                           cu.scale.data_ptr(), self._stream(dev))
        if rc:
            _call(rc)
        return out, cg, cu

    def backward(self, dh, gate, up, recompute: bool = False, stream=None):
        """(dgate, dup), and h again with recompute; gate and up both tensors
        or both Checkpoints."""
        dev = dh.get_device()
        if stream is not None or dev != self._device():
            return self._elsewhere(GatedAct.backward, dh, stream, (dh, gate, up, recompute))
        pd = self._ptr(dh, self._out, "dh", dev)
        if isinstance(gate, tuple) != isinstance(up, tuple):
            _invalid("gate and up are either two tensors or two Checkpoints")
        if isinstance(gate, tuple):
            saved = (None, None, *self._saved(gate, "gate", dev), *self._saved(up, "up", dev))
        else:
            saved = (self._ptr(gate, self._in, "gate", dev), self._ptr(up, self._in, "up", dev), None, None, None,
                     None)
        device = dh.device
        if self._halves:
            both = self._new((self.rows, self.in_pitch), dtype=self._torch_dtype, device=device)
            dgate = both.as_strided(self._shape, self._in)
            dup = both.as_strided(self._shape, self._in, self.cols)
        else:
            dgate, dup = self._empty(device, self.in_pitch), self._empty(device, self.in_pitch)
        h = self._empty(device, self.out_pitch) if recompute else None
        rc = tsx_gated_act_backward(*self._head, pd, *saved, dgate.data_ptr(), dup.data_ptr(),
                                    h.data_ptr() if recompute else None, self._stream(dev))
        if rc:
            _call(rc)
        return (dgate, dup, h) if recompute else (dgate, dup)


class GroupNorm(_Layer):
    """act(group norm of x) over [n, l, c], channels last (tsx_group_norm and
    its backward pass).  weight and bias [c] are fp32, or of the element type
    with param_dtype.  x_pitch: elements between the rows of x and dx; y_pitch:
    of y and dy."""

    def __init__(self, dtype: str, n: int, l: int, c: int, groups: int, act: str = "none", eps: float = 1e-5,
                 param_dtype: str = "f32", form: str = "int8", block: int = 128, x_pitch: int | None = None,
                 y_pitch: int | None = None):
        super().__init__(dtype, int(n) * int(l), c, form, block)
        self.n, self.l, self.groups, self.act = int(n), int(l), int(groups), act
        self.x_pitch = self.cols if x_pitch is None else int(x_pitch)
        self.y_pitch = self.cols if y_pitch is None else int(y_pitch)
        self._shape = (self.n, self.l, self.cols)
        self._x, self._y = self._strides_of(self.x_pitch), self._strides_of(self.y_pitch)
        self._channels, self._stats = (self.cols,), (self.n, self.groups)
        self._desc = tsx_norm_desc(self._dtype_code, _named(DTYPES, param_dtype, "param_dtype"),
                                   _named(ACTS, act, "activation"), self.groups, self._form_code, self.block, self.n,
                                   self.l, self.cols, self.x_pitch, self.y_pitch, eps)
        t = self._torch
        self._param = {"f16": t.float16, "bf16": t.bfloat16, "f32": t.float32}[param_dtype]
        self._ref = ctypes.byref(self._desc)
        # bytes of scratch, forward and backward, for tensors of any alignment and for aligned ones
        self._scratch = [[self._workspace(backward, aligned) for aligned in (0, 1)] for backward in (0, 1)]

    def _workspace(self, backward: int, aligned: int) -> int:
        size = ctypes.c_size_t()
        _call(tsx_group_norm_workspace(self._ref, backward, aligned, ctypes.byref(size)))
        return size.value

    def forward(self, x, weight, bias, out=None, checkpoint: bool = False, stream=None):
        """(y, mean, rstd), and with checkpoint x's Checkpoint too."""
        dev = x.get_device()
        if stream is not None or dev != self._device():
            return self._elsewhere(GroupNorm.forward, x, stream, (x, weight, bias, out, checkpoint))
        f32 = self._f32
        px = self._ptr(x, self._x, "x", dev)
        pw = self._vector(weight, self._channels, self._param, "weight", dev)
        pb = self._vector(bias, self._channels, self._param, "bias", dev)
        if out is None:
            out = self._empty(x.device, self.y_pitch)
            py = out.data_ptr()
        else:
            py = self._ptr(out, self._y, "out", dev)
        new, device = self._new, x.device
        mean, rstd = new(self._stats, dtype=f32, device=device), new(self._stats, dtype=f32, device=device)
        if checkpoint:
            saved = self._new_checkpoint(device)
            pq, ps = saved.q.data_ptr(), saved.scale.data_ptr()
        else:
            pq = ps = None
        size = self._scratch[0][not (px | py | (pq or 0)) & 15]
        scratch = new((size,), dtype=self._byte, device=device) if size else None
        rc = tsx_group_norm(self._ref, px, pw, pb, py, mean.data_ptr(), rstd.data_ptr(), pq, ps,
                            scratch.data_ptr() if size else None, size, self._stream(dev))
        if rc:
            _call(rc)
        return (out, mean, rstd, saved) if checkpoint else (out, mean, rstd)

    def backward(self, dy, saved, weight, bias, mean, rstd, out=None, stream=None):
        """(dx, dweight, dbias); saved: x or its Checkpoint."""
        dev = dy.get_device()
        if stream is not None or dev != self._device():
            return self._elsewhere(GroupNorm.backward, dy, stream, (dy, saved, weight, bias, mean, rstd, out))
        f32 = self._f32
        pdy = self._ptr(dy, self._y, "dy", dev)
        if isinstance(saved, tuple):
            src = (None, *self._saved(saved, "saved", dev))
        else:
            src = (self._ptr(saved, self._x, "saved", dev), None, None)
        pw = self._vector(weight, self._channels, self._param, "weight", dev)
        pb = self._vector(bias, self._channels, self._param, "bias", dev)
        pm = self._vector(mean, self._stats, f32, "mean", dev)
        pr = self._vector(rstd, self._stats, f32, "rstd", dev)
        if out is None:
            out = self._empty(dy.device, self.x_pitch)
            pdx = out.data_ptr()
        else:
            pdx = self._ptr(out, self._x, "out", dev)
        new, device = self._new, dy.device
        dweight, dbias = new(self._channels, dtype=f32, device=device), new(self._channels, dtype=f32, device=device)
        size = self._scratch[1][not (pdy | pdx | (src[0] or src[1] or 0)) & 15]
        scratch = new((size,), dtype=self._byte, device=device)
        rc = tsx_group_norm_backward(self._ref, pdy, *src, pw, pb, pm, pr, pdx, dweight.data_ptr(), dbias.data_ptr(),
                                     scratch.data_ptr(), size, self._stream(dev))
        if rc:
            _call(rc)
        return out, dweight, dbias
