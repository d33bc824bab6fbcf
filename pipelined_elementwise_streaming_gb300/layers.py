"""The layer operators of libtsx (include/tsx_layers.h) for torch tensors.

``GroupNorm``, ``GatedAct`` and ``Packer`` hold a shape and what the C calls
need of it; they own no device memory and may be used from several streams::

    norm = GroupNorm("bf16", n, l, c, groups=32, act="silu")
    y, mean, rstd, saved = norm.forward(x, weight, bias, checkpoint=True)
    dx, dweight, dbias = norm.backward(dy, saved, weight, bias, mean, rstd)

    glu = GatedAct("bf16", rows, cols, act="silu", in_pitch=2 * cols)
    h, gate8, up8 = glu.forward(both[:, :cols], both[:, cols:], checkpoint=True)
    dgate, dup = glu.backward(dh, gate8, up8)

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
    lib.tsx_group_norm_workspace.argtypes = [d, i, ctypes.POINTER(ctypes.c_size_t)]
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
        _invalid(f"unknown {what} {key!r}: one of {', '.join(table)}")
    return table[key]


class _Layer:
    """What the layers share: their torch types, the checks of tensors, and
    where results live."""

    def __init__(self, dtype: str, rows: int, cols: int, form: str, block: int):
        import torch

        self._torch = torch
        self._dtype_code = _named(DTYPES, dtype, "dtype")
        self._form_code = _named(FORMS, form, "8-bit form")
        self.dtype, self.rows, self.cols, self.form, self.block = dtype, int(rows), int(cols), form, int(block)
        self._torch_dtype = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self._q_dtype = torch.int8 if form == "int8" else torch.float8_e4m3fn
        if self.block not in (32, 64, 128):
            _invalid("block must be 32, 64 or 128")
        self._blocks = -(-self.cols // self.block)

    def _rows(self, t, pitch: int, name: str, device, shape=None) -> int:
        """The address of t as [rows, cols] of the element type with this row
        pitch, on `device`."""
        if t.dtype is not self._torch_dtype or t.device != device:
            _invalid(f"{name} must be a {self.dtype} tensor on {device}, got {t.dtype} on {t.device}")
        if tuple(t.shape) != (shape or (self.rows, self.cols)):
            _invalid(f"{name} must have shape {list(shape or (self.rows, self.cols))}, got {list(t.shape)}")
        if t.numel():
            stride, size = t.stride(), t.shape
            fits = stride[-1] == 1 or size[-1] == 1
            step = pitch
            for k in range(len(size) - 2, -1, -1):
                fits = fits and (stride[k] == step or size[k] == 1)
                step *= size[k]
            if not fits:
                _invalid(f"{name} must have a row pitch of {pitch} elements, got strides {list(stride)}")
        return t.data_ptr()

    def _saved(self, c: Checkpoint, name: str, device):
        q, scale = c
        if (q.dtype is not self._q_dtype or scale.dtype is not self._torch.float32 or q.device != device
                or scale.device != device):
            _invalid(f"{name} must be an {self.form} checkpoint with fp32 scales on {device}")
        if (tuple(q.shape) != (self.rows, self.cols) or tuple(scale.shape) != (self.rows, self._blocks)
                or not q.is_contiguous() or not scale.is_contiguous()):
            _invalid(f"{name} must hold dense [{self.rows}, {self.cols}] numbers and [{self.rows}, {self._blocks}] "
                     "scales")
        return q.data_ptr(), scale.data_ptr()

    def _vector(self, t, count: int, dtype, name: str, device) -> int:
        if t.dtype is not dtype or t.device != device or t.numel() != count or not t.is_contiguous():
            _invalid(f"{name} must be {count} contiguous {dtype} values on {device}")
        return t.data_ptr()

    def _empty(self, pitch: int, device, shape=None):
        t = self._torch
        if pitch == self.cols:
            return t.empty(shape or (self.rows, self.cols), dtype=self._torch_dtype, device=device)
        wide = t.empty(*(shape or (self.rows, self.cols))[:-1], pitch, dtype=self._torch_dtype, device=device)
        return wide[..., : self.cols]

    def _new_checkpoint(self, device) -> Checkpoint:
        t = self._torch
        return Checkpoint(t.empty(self.rows, self.cols, dtype=self._q_dtype, device=device),
                          t.empty(self.rows, self._blocks, dtype=t.float32, device=device))

    def _on(self, first, stream):
        """Run on the tensor's device, and allocate for the stream used."""
        if not first.is_cuda:
            _invalid("tensors must be on a CUDA device")
        return _Where(self._torch, first.device, stream)


class _Where:
    """The device and stream of one call, made current for its length only
    where they are not."""

    def __init__(self, torch, device, stream):
        self.device = device
        self._device = None if torch.cuda.current_device() == device.index else torch.cuda.device(device)
        self._stream = None if stream is None else torch.cuda.stream(stream)
        self._torch, self.handle = torch, stream.cuda_stream if stream is not None else None

    def __enter__(self):
        if self._device is not None:
            self._device.__enter__()
        if self._stream is not None:
            self._stream.__enter__()
        else:
            self.handle = self._torch.cuda.current_stream(self.device).cuda_stream
        return self

    def __exit__(self, *exc):
        if self._stream is not None:
            self._stream.__exit__(*exc)
        if self._device is not None:
            self._device.__exit__(*exc)


class Packer(_Layer):
    """Tensors [rows, cols] to 8 bits and back (tsx_pack, tsx_unpack)."""

    def __init__(self, dtype: str, rows: int, cols: int, form: str = "int8", block: int = 128,
                 pitch: int | None = None):
        super().__init__(dtype, rows, cols, form, block)
        self.pitch = self.cols if pitch is None else int(pitch)
        self._head = (self._dtype_code, self.rows, self.cols, self.pitch, self._form_code, self.block)

    def pack(self, x, out: Checkpoint | None = None, stream=None) -> Checkpoint:
        with self._on(x, stream) as w:
            px = self._rows(x, self.pitch, "x", w.device)
            out = self._new_checkpoint(w.device) if out is None else out
            _call(tsx_pack(*self._head, px, *self._saved(out, "out", w.device), w.handle))
        return out

    def unpack(self, saved: Checkpoint, out=None, stream=None):
        with self._on(saved.q, stream) as w:
            pq = self._saved(saved, "saved", w.device)
            out = self._empty(self.pitch, w.device) if out is None else out
            _call(tsx_unpack(*self._head, *pq, self._rows(out, self.pitch, "out", w.device), w.handle))
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
        self._head = (self._dtype_code, self.rows, self.cols, self.in_pitch, self.out_pitch,
                      _named(ACTS, act, "activation"), self._form_code, self.block)

    def forward(self, gate, up, out=None, checkpoint: bool = False, stream=None):
        """h, or with checkpoint (h, gate's Checkpoint, up's Checkpoint)."""
        with self._on(gate, stream) as w:
            pg = self._rows(gate, self.in_pitch, "gate", w.device)
            pu = self._rows(up, self.in_pitch, "up", w.device)
            out = self._empty(self.out_pitch, w.device) if out is None else out
            ph = self._rows(out, self.out_pitch, "out", w.device)
            if not checkpoint:
                _call(tsx_gated_act(*self._head, pg, pu, ph, None, None, None, None, w.handle))
                return out
            cg, cu = self._new_checkpoint(w.device), self._new_checkpoint(w.device)
            _call(tsx_gated_act(*self._head, pg, pu, ph, cg.q.data_ptr(), cg.scale.data_ptr(), cu.q.data_ptr(),
                                cu.scale.data_ptr(), w.handle))
            return out, cg, cu

    def backward(self, dh, gate, up, recompute: bool = False, stream=None):
        """(dgate, dup), and h again with recompute; gate and up both tensors
        or both Checkpoints."""
        with self._on(dh, stream) as w:
            pd = self._rows(dh, self.out_pitch, "dh", w.device)
            if isinstance(gate, tuple) != isinstance(up, tuple):
                _invalid("gate and up are either two tensors or two Checkpoints")
            if isinstance(gate, tuple):
                saved = (None, None, *self._saved(gate, "gate", w.device), *self._saved(up, "up", w.device))
            else:
                saved = (self._rows(gate, self.in_pitch, "gate", w.device),
                         self._rows(up, self.in_pitch, "up", w.device), None, None, None, None)
            if self.in_pitch >= 2 * self.cols:
                both = self._torch.empty(self.rows, self.in_pitch, dtype=self._torch_dtype, device=w.device)
                dgate, dup = both[:, : self.cols], both[:, self.cols: 2 * self.cols]
            else:
                dgate, dup = self._empty(self.in_pitch, w.device), self._empty(self.in_pitch, w.device)
            h = self._empty(self.out_pitch, w.device) if recompute else None
            _call(tsx_gated_act_backward(*self._head, pd, *saved, dgate.data_ptr(), dup.data_ptr(),
                                         h.data_ptr() if recompute else None, w.handle))
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
        self._param = {"f16": self._torch.float16, "bf16": self._torch.bfloat16, "f32": self._torch.float32}.get(
            param_dtype)
        self._desc = tsx_norm_desc(self._dtype_code, _named(DTYPES, param_dtype, "param_dtype"),
                                   _named(ACTS, act, "activation"), self.groups, self._form_code, self.block, self.n,
                                   self.l, self.cols, self.x_pitch, self.y_pitch, eps)
        self._ref = ctypes.byref(self._desc)
        self._scratch = []
        for backward in (0, 1):
            size = ctypes.c_size_t()
            _call(tsx_group_norm_workspace(self._ref, backward, ctypes.byref(size)))
            self._scratch.append(size.value)

    def _params(self, weight, bias, device):
        return (self._vector(weight, self.cols, self._param, "weight", device),
                self._vector(bias, self.cols, self._param, "bias", device))

    def forward(self, x, weight, bias, out=None, checkpoint: bool = False, stream=None):
        """(y, mean, rstd), and with checkpoint x's Checkpoint too."""
        t = self._torch
        with self._on(x, stream) as w:
            px = self._rows(x, self.x_pitch, "x", w.device, self._shape)
            pw, pb = self._params(weight, bias, w.device)
            out = self._empty(self.y_pitch, w.device, self._shape) if out is None else out
            py = self._rows(out, self.y_pitch, "out", w.device, self._shape)
            mean, rstd = t.empty(2, self.n, self.groups, dtype=t.float32, device=w.device)
            scratch = t.empty(self._scratch[0], dtype=t.uint8, device=w.device)
            saved = self._new_checkpoint(w.device) if checkpoint else None
            pq, ps = (saved.q.data_ptr(), saved.scale.data_ptr()) if checkpoint else (None, None)
            _call(tsx_group_norm(self._ref, px, pw, pb, py, mean.data_ptr(), rstd.data_ptr(), pq, ps,
                                 scratch.data_ptr(), self._scratch[0], w.handle))
        return (out, mean, rstd, saved) if checkpoint else (out, mean, rstd)

    def backward(self, dy, saved, weight, bias, mean, rstd, out=None, stream=None):
        """(dx, dweight, dbias); saved: x or its Checkpoint."""
        t = self._torch
        with self._on(dy, stream) as w:
            pdy = self._rows(dy, self.y_pitch, "dy", w.device, self._shape)
            if isinstance(saved, tuple):
                src = (None, *self._saved(saved, "saved", w.device))
            else:
                src = (self._rows(saved, self.x_pitch, "saved", w.device, self._shape), None, None)
            pw, pb = self._params(weight, bias, w.device)
            pm = self._vector(mean, self.n * self.groups, t.float32, "mean", w.device)
            pr = self._vector(rstd, self.n * self.groups, t.float32, "rstd", w.device)
            out = self._empty(self.x_pitch, w.device, self._shape) if out is None else out
            pdx = self._rows(out, self.x_pitch, "out", w.device, self._shape)
            dweight, dbias = t.empty(2, self.cols, dtype=t.float32, device=w.device)
            scratch = t.empty(self._scratch[1], dtype=t.uint8, device=w.device)
            _call(tsx_group_norm_backward(self._ref, pdy, *src, pw, pb, pm, pr, pdx, dweight.data_ptr(),
                                          dbias.data_ptr(), scratch.data_ptr(), self._scratch[1], w.handle))
        return out, dweight, dbias
