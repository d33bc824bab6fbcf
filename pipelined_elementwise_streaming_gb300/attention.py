"""The operators around attention of libtsx (include/tsx_attention.h) for torch
tensors.

``Rotary`` turns queries and keys to their positions, with a norm of each head
in the same pass if asked to; ``PagedAttention`` appends keys and values to a
paged cache, turned on the way, and attends over it::

    rope = Rotary("bf16", q_heads, k_heads, dim, norm="rms")
    q2, k2 = rope.forward(q, k, positions, q_weight, k_weight)
    dq, dk, dq_weight, dk_weight = rope.backward(dq2, dk2, positions, q, k, q_weight, k_weight)

    attention = PagedAttention("bf16", q_heads, k_heads, dim, page_size=16, rotary=rope)
    cache = attention.new_cache(pages)
    batch = Batch(starts, lengths, pages_of, most_new)
    q2 = attention.append(q, k, v, cache, batch, q_weight, k_weight)
    out = attention.forward(q2, cache, batch)

Queries, keys and values are [tokens, heads, dim] with any pitches that keep
heads apart (the slices of one projection, say); the objects hold no tokens and
no device memory and may be used from several streams and threads.

Autograd does not see the calls: what they return has no graph, also for inputs
that require gradients.  Results and scratch come from torch's allocator for the
stream that the call runs on; tensors that the caller passes with ``stream=``
belong to the caller, who keeps them alive until that stream's work is done.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

from . import DTYPES, lib
from .layers import _call, _invalid, _Layer, _named

LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}
NORMS = {None: 0, "rms": 1}


class tsx_heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("pitch", ctypes.c_int64), ("head_pitch", ctypes.c_int64)]


class tsx_rotary_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "param_dtype", "q_heads", "k_heads", "dim", "rot", "layout",
                                              "norm")] + \
               [("eps", ctypes.c_float), ("amplitude", ctypes.c_float), ("turns", ctypes.c_uint64 * 128)]


class tsx_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "heads", "dim", "page_size")] + \
               [(n, ctypes.c_int64) for n in ("pages", "page_pitch", "slot_pitch", "head_pitch")] + \
               [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]


class tsx_batch(ctypes.Structure):
    _fields_ = [("starts", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("pages", ctypes.c_void_p),
                ("pages_pitch", ctypes.c_int64), ("seqs", ctypes.c_int32), ("most_pages", ctypes.c_int32)]


def _declare():
    p, i, i64, d = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double
    size = ctypes.POINTER(ctypes.c_size_t)
    lib.tsx_rotary_frequencies.argtypes = [i, d, i, d, d, d, d, p, ctypes.POINTER(ctypes.c_float)]
    lib.tsx_rotary_turns.argtypes = [i, p, p]
    # structures by address: ctypes.byref, or None
    lib.tsx_rotary.argtypes = [p, i64, p, i] + [p] * 7
    lib.tsx_rotary_workspace.argtypes = [p, i64, size]
    lib.tsx_rotary_backward.argtypes = [p, i64, p, i] + [p] * 11 + [ctypes.c_size_t, p]
    lib.tsx_cache_append.argtypes = [p, p, p, i64] + [p] * 7
    lib.tsx_paged_attention_workspace.argtypes = [p, i64, i, i64, size]
    lib.tsx_paged_attention.argtypes = [p, p, i64, i, i64, ctypes.c_float, p, p, p, p, ctypes.c_size_t, p]


_declare()

tsx_rotary_frequencies = lib.tsx_rotary_frequencies
tsx_rotary_turns = lib.tsx_rotary_turns
tsx_rotary = lib.tsx_rotary
tsx_rotary_workspace = lib.tsx_rotary_workspace
tsx_rotary_backward = lib.tsx_rotary_backward
tsx_cache_append = lib.tsx_cache_append
tsx_paged_attention_workspace = lib.tsx_paged_attention_workspace
tsx_paged_attention = lib.tsx_paged_attention

_ref = ctypes.byref


class Batch(NamedTuple):
    """Sequences with new tokens (tsx_batch): int32 CUDA tensors starts
    [seqs + 1], lengths [seqs] (with the new tokens) and pages [seqs, most
    pages of a sequence], and the most new tokens that one of them has, as far
    as the host knows (it only chooses between kernels)."""
    starts: object
    lengths: object
    pages: object
    most_new: int


class _Heads(_Layer):
    """What the operators on [tokens, heads, dim] share."""

    def __init__(self, dtype: str, q_heads: int, k_heads: int, dim: int):
        import torch

        self._torch = torch
        self._dtype_code = _named(DTYPES, dtype, "dtype")
        self.dtype, self.q_heads, self.k_heads, self.dim = dtype, int(q_heads), int(k_heads), int(dim)
        if self.q_heads < 0 or self.k_heads < 0 or not 1 <= self.dim <= 256:
            _invalid("heads must not be negative, and dim must be 1 .. 256")
        self._torch_dtype = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self._f32, self._byte, self._i32, self._i64 = torch.float32, torch.uint8, torch.int32, torch.int64
        self._device = torch._C._cuda_getDevice
        self._stream = torch._C._cuda_getCurrentRawStream
        self._new = torch.empty

    def _tensor(self, t, tokens: int, heads: int, name: str, dev: int):
        """t as the C calls take it; None for a tensor without heads."""
        if t is None:
            if heads:
                _invalid(f"{name} is required")
            return None
        if t.dtype is not self._torch_dtype or t.get_device() != dev:
            _invalid(f"{name} must be a {self.dtype} tensor on cuda:{dev}, got {t.dtype} on {t.device}")
        if t.shape != (tokens, heads, self.dim):
            _invalid(f"{name} must have shape {[tokens, heads, self.dim]}, got {list(t.shape)}")
        pitch, head, one = t.stride()
        if one != 1 and self.dim > 1 and t.numel():
            _invalid(f"{name} must have its channels side by side, got strides {list(t.stride())}")
        return tsx_heads(t.data_ptr(), pitch, head)

    def _result(self, out, like, tokens: int, heads: int, name: str, dev: int):
        """(out or a new dense tensor, as the C calls take it)"""
        if out is None:
            out = self._new((tokens, heads, self.dim), dtype=self._torch_dtype, device=like.device)
            return out, tsx_heads(out.data_ptr(), heads * self.dim, self.dim)
        return out, self._tensor(out, tokens, heads, name, dev)

    def _tokens(self, t, name: str) -> int:
        if t is None or t.dim() != 3:
            _invalid(f"{name} must be a tensor [tokens, heads, dim]")
        return t.shape[0]


def _addr(s):
    return None if s is None else _ref(s)


class Rotary(_Heads):
    """Rotary positions of queries [tokens, q_heads, dim] and keys [tokens,
    k_heads, dim] (tsx_rotary and its backward pass).

    rot: how many channels of a head turn (all by default).  layout: "half"
    (channel i with i + rot / 2) or "interleaved" (2 i with 2 i + 1).
    Frequencies: base^(-2 i / rot), scaled as `scaling` says, None, ("linear",
    factor), ("ntk", factor) or ("yarn", factor, length of training[, fast,
    slow]); or `frequencies`, rot / 2 numbers in radians to a position, and
    `amplitude`.  norm="rms" norms each head before the rotation; the weights
    are fp32, or of the element type with param_dtype."""

    def __init__(self, dtype: str, q_heads: int, k_heads: int, dim: int, rot: int | None = None,
                 layout: str = "half", base: float = 10000.0, scaling=None, frequencies=None,
                 amplitude: float | None = None, norm: str | None = None, eps: float = 1e-6,
                 param_dtype: str = "f32"):
        super().__init__(dtype, q_heads, k_heads, dim)
        t = self._torch
        self.rot = self.dim if rot is None else int(rot)
        if self.rot % 2 or not 0 <= self.rot <= self.dim:
            _invalid("rot must be even, 0 .. dim")
        self.layout, self.norm, self.eps = layout, norm, float(eps)
        table = (ctypes.c_double * 128)()
        if frequencies is None:
            kind, *numbers = (None,) if scaling is None else (scaling,) if isinstance(scaling, str) else scaling
            code = _named(SCALINGS, kind, "scaling")
            least, most = ((0, 0), (1, 1), (1, 1), (2, 4))[code]
            if not least <= len(numbers) <= most:
                _invalid(f"scaling {kind!r} takes {least} to {most} numbers")
            factor, length, fast, slow = [float(v) for v in numbers] + [1.0, 1.0, 32.0, 1.0][len(numbers):]
            grown = ctypes.c_float()
            _call(tsx_rotary_frequencies(self.rot, float(base), code, factor, length, fast, slow, table, _ref(grown)))
            if amplitude is None:
                amplitude = grown.value
        else:
            if scaling is not None:
                _invalid("scaling belongs to frequencies of a base")
            values = [float(v) for v in frequencies]
            if len(values) != self.rot // 2:
                _invalid(f"there must be {self.rot // 2} frequencies, one to a pair")
            table[: len(values)] = values
        self.frequencies = tuple(table[: self.rot // 2])
        self.amplitude = 1.0 if amplitude is None else float(amplitude)
        self._desc = tsx_rotary_desc(self._dtype_code, _named(DTYPES, param_dtype, "param_dtype"), self.q_heads,
                                     self.k_heads, self.dim, self.rot, _named(LAYOUTS, layout, "layout"),
                                     _named(NORMS, norm, "norm"), self.eps, self.amplitude)
        _call(tsx_rotary_turns(self.rot // 2, table, self._desc.turns))
        self._param = {"f16": t.float16, "bf16": t.bfloat16, "f32": t.float32}[param_dtype]
        self._ref = _ref(self._desc)
        # bytes of scratch do not depend on how many tokens there are; the description is checked on the way
        size = ctypes.c_size_t()
        _call(tsx_rotary_workspace(self._ref, 1, _ref(size)))
        self._scratch = size.value

    def _positions(self, positions, tokens: int, dev: int):
        if positions.dtype is not self._i64 and positions.dtype is not self._i32 or positions.get_device() != dev:
            _invalid(f"positions must be int64 or int32 on cuda:{dev}, got {positions.dtype} on {positions.device}")
        if positions.shape != (tokens,) or (tokens > 1 and positions.stride(0) != 1):
            _invalid(f"positions must be {tokens} contiguous numbers, got {list(positions.shape)}")
        return positions.data_ptr(), 8 if positions.dtype is self._i64 else 4

    def _weight(self, w, name: str, dev: int):
        if w is None:
            return None
        if self.norm is None:
            _invalid(f"{name} belongs to a norm")
        return self._vector(w, (self.dim,), self._param, name, dev)

    def forward(self, q, k, positions, q_weight=None, k_weight=None, q_out=None, k_out=None, stream=None):
        """(q, k) turned, new tensors or q_out and k_out.  k is None where
        there are no k_heads (q where there are no q_heads), and so is its
        result."""
        first = q if q is not None else k
        tokens = self._tokens(first, "q" if q is not None else "k")
        dev = first.get_device()
        if stream is not None or dev != self._device():
            return self._elsewhere(Rotary.forward, first, stream, (q, k, positions, q_weight, k_weight, q_out, k_out))
        tq = self._tensor(q, tokens, self.q_heads, "q", dev)
        tk = self._tensor(k, tokens, self.k_heads, "k", dev)
        at, wide = self._positions(positions, tokens, dev)
        wq, wk = self._weight(q_weight, "q_weight", dev), self._weight(k_weight, "k_weight", dev)
        rq = rk = None
        if tq is not None:
            q_out, rq = self._result(q_out, first, tokens, self.q_heads, "q_out", dev)
        if tk is not None:
            k_out, rk = self._result(k_out, first, tokens, self.k_heads, "k_out", dev)
        rc = tsx_rotary(self._ref, tokens, at, wide, _addr(tq), _addr(tk), wq, wk, _addr(rq), _addr(rk),
                        self._stream(dev))
        if rc:
            _call(rc)
        return q_out, k_out

    def backward(self, dq, dk, positions, q=None, k=None, q_weight=None, k_weight=None, q_out=None, k_out=None,
                 stream=None):
        """(dq, dk) of the inputs from those of the results; with a norm, which
        needs the inputs q and k, (dq, dk, dq_weight, dk_weight), a weight's
        gradient None where the weight is."""
        first = dq if dq is not None else dk
        tokens = self._tokens(first, "dq" if dq is not None else "dk")
        dev = first.get_device()
        if stream is not None or dev != self._device():
            return self._elsewhere(Rotary.backward, first, stream,
                                   (dq, dk, positions, q, k, q_weight, k_weight, q_out, k_out))
        tdq = self._tensor(dq, tokens, self.q_heads, "dq", dev)
        tdk = self._tensor(dk, tokens, self.k_heads, "dk", dev)
        at, wide = self._positions(positions, tokens, dev)
        wq, wk = self._weight(q_weight, "q_weight", dev), self._weight(k_weight, "k_weight", dev)
        tq = tk = rq = rk = None
        if self.norm is not None:
            tq = self._tensor(q, tokens, self.q_heads, "q", dev)
            tk = self._tensor(k, tokens, self.k_heads, "k", dev)
        elif q is not None or k is not None:
            _invalid("q and k belong to the gradient of a norm")
        if tdq is not None:
            q_out, rq = self._result(q_out, first, tokens, self.q_heads, "q_out", dev)
        if tdk is not None:
            k_out, rk = self._result(k_out, first, tokens, self.k_heads, "k_out", dev)
        new, device = self._new, first.device
        gq = None if wq is None else new((self.dim,), dtype=self._f32, device=device)
        gk = None if wk is None else new((self.dim,), dtype=self._f32, device=device)
        scratch = None
        if gq is not None or gk is not None:
            scratch = new((self._scratch,), dtype=self._byte, device=device)
        rc = tsx_rotary_backward(self._ref, tokens, at, wide, _addr(tdq), _addr(tdk), _addr(tq), _addr(tk), wq, wk,
                                 _addr(rq), _addr(rk), None if gq is None else gq.data_ptr(),
                                 None if gk is None else gk.data_ptr(), None if scratch is None else scratch.data_ptr(),
                                 self._scratch if scratch is not None else 0, self._stream(dev))
        if rc:
            _call(rc)
        return (q_out, k_out) if self.norm is None else (q_out, k_out, gq, gk)


class PagedAttention(_Heads):
    """A paged cache of keys and values and attention over it
    (tsx_cache_append, tsx_paged_attention).

    A cache is two tensors (keys, values) [pages, page_size, kv_heads, dim] of
    the same strides, dim side by side (``new_cache`` makes them; heads before
    slots is a permuted view).  rotary: the ``Rotary`` that turns (and norms)
    queries and keys as they come in, or None to append them as they are.
    scale: of the scores, 1 / sqrt(dim) by default."""

    def __init__(self, dtype: str, q_heads: int, kv_heads: int, dim: int, page_size: int, rotary: Rotary | None = None,
                 scale: float | None = None):
        super().__init__(dtype, q_heads, kv_heads, dim)
        self.page_size, self.rotary = int(page_size), rotary
        if not 1 <= self.page_size <= 1 << 20:
            _invalid("page_size must be 1 .. 2^20")
        if self.k_heads < 1 or self.q_heads < 1 or self.q_heads % self.k_heads:
            _invalid("q_heads must be a multiple of kv_heads, and both above 0")
        self.scale = self.dim ** -0.5 if scale is None else float(scale)
        if not abs(self.scale) <= 2.0**127:
            _invalid("scale must be finite, 2^127 at most")
        self._scratch = {}
        if rotary is None:
            self._rope = Rotary(dtype, q_heads, kv_heads, dim, rot=0)
        elif (rotary.dtype, rotary.q_heads, rotary.k_heads, rotary.dim) != (dtype, self.q_heads, self.k_heads, self.dim):
            _invalid("the rotary's dtype, heads and dim must be the attention's")
        else:
            self._rope = rotary

    def new_cache(self, pages: int, device=None):
        """(keys, values) of this many pages, zeros."""
        shape = (int(pages), self.page_size, self.k_heads, self.dim)
        device = self._torch.device("cuda") if device is None else device
        return tuple(self._torch.zeros(shape, dtype=self._torch_dtype, device=device) for _ in range(2))

    def _cache(self, cache, dev: int) -> tsx_cache:
        k, v = cache
        dt, shape, strides = self._torch_dtype, k.shape, k.stride()
        if (len(shape) == 4 and shape == v.shape and strides == v.stride() and k.dtype is dt and v.dtype is dt
                and k.get_device() == dev and v.get_device() == dev):   # as a rule; else what is wrong
            pages, slots, heads, dim = shape
            if slots == self.page_size and heads == self.k_heads and dim == self.dim and (strides[3] == 1 or dim == 1):
                return tsx_cache(self._dtype_code, heads, dim, slots, pages, strides[0], strides[1], strides[2],
                                 k.data_ptr(), v.data_ptr())
        if k.dtype is not dt or v.dtype is not dt or k.get_device() != dev or v.get_device() != dev:
            _invalid(f"the cache must be two {self.dtype} tensors on cuda:{dev}")
        if len(shape) != 4 or shape[1:] != (self.page_size, self.k_heads, self.dim) or v.shape != shape:
            _invalid(f"keys and values must have shape [pages, {self.page_size}, {self.k_heads}, {self.dim}], got "
                     f"{list(shape)} and {list(v.shape)}")
        _invalid("keys and values must have the same strides, and channels side by side")

    def _batch(self, batch: Batch, dev: int) -> tsx_batch:
        starts, lengths, pages, _ = batch
        i32 = self._i32
        if (starts.dtype is not i32 or lengths.dtype is not i32 or pages.dtype is not i32
                or starts.get_device() != dev or lengths.get_device() != dev or pages.get_device() != dev):
            _invalid(f"starts, lengths and pages must be int32 tensors on cuda:{dev}")
        shape, strides, seqs = pages.shape, pages.stride(), lengths.numel()
        if len(shape) != 2 or shape[0] != seqs or lengths.dim() != 1 or starts.shape != (seqs + 1,):
            _invalid("starts must be [seqs + 1], lengths [seqs] and pages [seqs, most pages of a sequence]")
        if not starts.is_contiguous() or not lengths.is_contiguous() or (strides[1] != 1 and shape[1] > 1):
            _invalid("starts, lengths and each sequence's pages must be contiguous")
        return tsx_batch(starts.data_ptr(), lengths.data_ptr(), pages.data_ptr(), strides[0], seqs, shape[1])

    def _workspace(self, cache: tsx_cache, most_new: int) -> int:
        """Bytes of scratch, which do not depend on the tokens; remembered for a
        few values of most_new."""
        size = ctypes.c_size_t()
        _call(tsx_paged_attention_workspace(_ref(cache), 1, self.q_heads, most_new, _ref(size)))
        if len(self._scratch) < 64:
            self._scratch[most_new] = size.value
        return size.value

    def append(self, q, k, v, cache, batch: Batch, q_weight=None, k_weight=None, out=None, stream=None):
        """Puts the new tokens' k and v into the cache and returns q turned (a
        new tensor or out).  Rows that belong to no sequence are left as they
        are, in a new tensor undefined.  q may be None: then so is the result,
        and k alone is turned."""
        tokens = self._tokens(k, "k")
        dev = k.get_device()
        if stream is not None or dev != self._device():
            return self._elsewhere(PagedAttention.append, k, stream, (q, k, v, cache, batch, q_weight, k_weight, out))
        rope = self._rope
        tk, tv = self._tensor(k, tokens, self.k_heads, "k", dev), self._tensor(v, tokens, self.k_heads, "v", dev)
        c, b = self._cache(cache, dev), self._batch(batch, dev)
        wq, wk = rope._weight(q_weight, "q_weight", dev), rope._weight(k_weight, "k_weight", dev)
        tq = to = None
        desc = rope._desc
        if q is None:
            desc = tsx_rotary_desc.from_buffer_copy(desc)
            desc.q_heads = 0
            wq = None
        else:
            tq = self._tensor(q, tokens, self.q_heads, "q", dev)
            out, to = self._result(out, k, tokens, self.q_heads, "out", dev)
        rc = tsx_cache_append(_ref(desc), _ref(c), _ref(b), tokens, _addr(tq), _ref(tk), _ref(tv), wq, wk, _addr(to),
                              self._stream(dev))
        if rc:
            _call(rc)
        return out

    def forward(self, q, cache, batch: Batch, out=None, lse: bool = False, stream=None):
        """softmax(scale q k^T) v over each token's sequence up to its own
        place, [tokens, q_heads, dim] (a new tensor or out; it may be q); with
        lse also the logs of the sums [tokens, q_heads] (fp32).  Rows that
        belong to no sequence are left as they are, in a new tensor
        undefined."""
        tokens = self._tokens(q, "q")
        dev = q.get_device()
        if stream is not None or dev != self._device():
            return self._elsewhere(PagedAttention.forward, q, stream, (q, cache, batch, out, lse))
        tq = self._tensor(q, tokens, self.q_heads, "q", dev)
        c, b = self._cache(cache, dev), self._batch(batch, dev)
        out, to = self._result(out, q, tokens, self.q_heads, "out", dev)
        logs = self._new((tokens, self.q_heads), dtype=self._f32, device=q.device) if lse else None
        most_new = int(batch.most_new)
        size = self._scratch.get(most_new)
        if size is None:
            size = self._workspace(c, most_new)
        scratch = self._new((size,), dtype=self._byte, device=q.device)
        rc = tsx_paged_attention(_ref(c), _ref(b), tokens, self.q_heads, most_new, self.scale, _ref(tq), _ref(to),
                                 None if logs is None else logs.data_ptr(), scratch.data_ptr(), size,
                                 self._stream(dev))
        if rc:
            _call(rc)
        return (out, logs) if lse else out
