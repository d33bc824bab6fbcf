"""The operators around attention on the host (no GPU): frequencies, what is
refused, scratch sizes, and the plain definitions against themselves."""

import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import attention as ref

A = 1 << 20   # stands for an address: calls that are refused look at no memory


@pytest.fixture(scope="module")
def tsx():
    import __graft_entry__

    __graft_entry__.build()
    import pipelined_elementwise_streaming_gb300 as m

    return m


# ------------------------------------------------------------ frequencies


@pytest.mark.parametrize("rot", [2, 8, 64, 126, 128, 256])
@pytest.mark.parametrize("scaling", [None, ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0, 4096), ("yarn", 4.0, 32768, 16, 2)])
def test_frequencies(tsx, rot, scaling):
    f = tsx.Rotary("bf16", 1, 1, 256, rot=rot, scaling=scaling, base=500000.0)
    want, amplitude = ref.frequencies(rot, base=500000.0, scaling=scaling)
    np.testing.assert_allclose(f.frequencies, want, rtol=1e-13)
    assert abs(f.amplitude - amplitude) <= 2.0**-24 * amplitude


def test_turns_are_the_part_of_a_turn(tsx):
    """To two units of 2^-64, over the range of frequencies."""
    rng = np.random.default_rng(0)
    values = [0.0, 1.0, 2 * math.pi, math.pi, 1e-9, 2.0**-40, 123.456, -0.25, -1.0, 2.0**30] + \
        list(np.exp(rng.uniform(-30, 5, 100)))
    table = (ctypes.c_double * len(values))(*values)
    out = (ctypes.c_uint64 * len(values))()
    assert tsx.tsx_rotary_turns(len(values), table, out) == tsx.TSX_OK
    # 2 pi to 60 digits
    tau = Fraction("6.28318530717958647692528676655900576839433879875021164194988918461563281257241799725606965")
    for v, got in zip(values, out):
        exact = Fraction(v) / tau * 2**64
        off = (got - exact) % 2**64
        # a unit or two, and the double-double quotient's 2^-100 of the value
        assert min(off, 2**64 - off) <= 2 + abs(exact) / 2**98, v


def test_frequencies_that_are_refused(tsx):
    good = dict(rot=64, base=1e4, scaling=0, factor=1.0, length=1.0, fast=32.0, slow=1.0)
    table, grown = (ctypes.c_double * 128)(), ctypes.c_float()
    for bad in (dict(rot=-2), dict(rot=63), dict(rot=258), dict(base=1.0), dict(base=float("inf")),
                dict(base=float("nan")), dict(scaling=4), dict(scaling=-1), dict(scaling=1, factor=0.5),
                dict(scaling=2, factor=float("nan")), dict(scaling=3, length=0.0), dict(scaling=3, slow=0.0),
                dict(scaling=3, fast=0.5)):
        args = dict(good, **bad)
        assert tsx.tsx_rotary_frequencies(*args.values(), table, ctypes.byref(grown)) == tsx.TSX_ERR_INVALID, bad
        assert tsx.tsx_last_error()
    assert tsx.tsx_rotary_frequencies(*good.values(), None, ctypes.byref(grown)) == tsx.TSX_ERR_INVALID
    assert tsx.tsx_rotary_frequencies(*good.values(), table, ctypes.byref(grown)) == tsx.TSX_OK
    out = (ctypes.c_uint64 * 128)()
    for v in (float("nan"), float("inf"), 2.0**31):
        table[0] = v
        assert tsx.tsx_rotary_turns(1, table, out) == tsx.TSX_ERR_INVALID
    assert tsx.tsx_rotary_turns(129, table, out) == tsx.TSX_ERR_INVALID
    assert tsx.tsx_rotary_turns(0, None, None) == tsx.TSX_OK


# ----------------------------------------------------------- constructors


def test_constructors(tsx):
    for make in (lambda: tsx.Rotary("f64", 1, 1, 64), lambda: tsx.Rotary("bf16", -1, 1, 64),
                 lambda: tsx.Rotary("bf16", 1, 1, 0), lambda: tsx.Rotary("bf16", 1, 1, 257),
                 lambda: tsx.Rotary("bf16", 1, 1, 64, rot=3), lambda: tsx.Rotary("bf16", 1, 1, 64, rot=66),
                 lambda: tsx.Rotary("bf16", 1, 1, 64, layout="other"),
                 lambda: tsx.Rotary("bf16", 1, 1, 64, norm="layer"),
                 lambda: tsx.Rotary("bf16", 1, 1, 64, eps=-1.0, norm="rms"),
                 lambda: tsx.Rotary("bf16", 1, 1, 64, eps=float("nan")),
                 lambda: tsx.Rotary("bf16", 1, 1, 64, param_dtype="f16"),
                 lambda: tsx.Rotary("bf16", 1, 1, 64, amplitude=float("inf")),
                 lambda: tsx.Rotary("bf16", 1, 1, 64, base=0.5),
                 lambda: tsx.Rotary("bf16", 1, 1, 64, scaling=("other", 2.0)),
                 lambda: tsx.Rotary("bf16", 1, 1, 64, scaling=("linear",)),
                 lambda: tsx.Rotary("bf16", 1, 1, 64, scaling=("yarn", 2.0)),
                 lambda: tsx.Rotary("bf16", 1, 1, 64, scaling=("linear", 0.1)),
                 lambda: tsx.Rotary("bf16", 1, 1, 64, frequencies=[1.0] * 31),
                 lambda: tsx.Rotary("bf16", 1, 1, 64, frequencies=[float("nan")] * 32),
                 lambda: tsx.Rotary("bf16", 1, 1, 64, frequencies=[1.0] * 32, scaling=("linear", 2.0)),
                 lambda: tsx.PagedAttention("bf16", 5, 2, 64, 16), lambda: tsx.PagedAttention("bf16", 4, 0, 64, 16),
                 lambda: tsx.PagedAttention("bf16", 0, 0, 64, 16), lambda: tsx.PagedAttention("bf16", 4, 2, 64, 0),
                 lambda: tsx.PagedAttention("bf16", 4, 2, 64, 1 << 21),
                 lambda: tsx.PagedAttention("bf16", 4, 2, 64, 16, scale=float("nan")),
                 lambda: tsx.PagedAttention("bf16", 4, 2, 64, 16, rotary=tsx.Rotary("f16", 4, 2, 64)),
                 lambda: tsx.PagedAttention("bf16", 4, 2, 64, 16, rotary=tsx.Rotary("bf16", 4, 4, 64))):
        with pytest.raises(tsx.TsxError) as e:
            make()
        assert e.value.code == tsx.TSX_ERR_INVALID and len(str(e.value)) > 15


class Fake:
    """A tensor on a device that no test has."""

    def __init__(self, device):
        import torch

        self.device, self.is_cuda, self.shape = torch.device("cuda", device), True, (4, 4, 64)

    def get_device(self):
        return self.device.index

    def dim(self):
        return 3


def test_a_stream_of_another_device_is_refused(tsx, monkeypatch):
    import types

    import torch

    stream = types.SimpleNamespace(device=torch.device("cuda", 1), device_index=1)
    x, rope = Fake(0), tsx.Rotary("bf16", 4, 4, 64)
    att = tsx.PagedAttention("bf16", 4, 4, 64, 16, rotary=rope)
    for op in (rope, att):
        monkeypatch.setattr(op, "_device", lambda: 0)
    batch = tsx.Batch(x, x, x, 1)
    for call in (lambda: rope.forward(x, x, x, stream=stream), lambda: rope.backward(x, x, x, stream=stream),
                 lambda: att.append(x, x, x, (x, x), batch, stream=stream),
                 lambda: att.forward(x, (x, x), batch, stream=stream)):
        with pytest.raises(tsx.TsxError) as e:
            call()
        assert e.value.code == tsx.TSX_ERR_INVALID and "cuda:1" in str(e.value)


def test_tensors_on_the_host_are_refused(tsx):
    import torch

    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    pos = torch.zeros(4, dtype=torch.int64)
    rope = tsx.Rotary("bf16", 4, 4, 64)
    att = tsx.PagedAttention("bf16", 4, 4, 64, 16)
    i32 = torch.zeros(2, dtype=torch.int32)
    for op in (rope, att):
        op._device = lambda: 0
    for call in (lambda: rope.forward(q, q, pos), lambda: att.forward(q, (q, q), tsx.Batch(i32, i32, i32, 1)),
                 lambda: rope.forward(None, None, pos), lambda: rope.forward(q[0], q, pos)):
        with pytest.raises(tsx.TsxError) as e:
            call()
        assert e.value.code == tsx.TSX_ERR_INVALID


# -------------------------------------------------------------- refusals


@pytest.fixture
def refused(tsx):
    import torch

    if torch.cuda.is_available():
        pytest.skip("stands-in for addresses stay off GPUs")

    def check(rc, code, word):
        assert rc == code and word in tsx.tsx_last_error(), (rc, tsx.tsx_last_error())

    return check


def heads(tsx, data=A, pitch=4096, head=128):
    return ctypes.byref(tsx.tsx_heads(data, pitch, head))


def desc(tsx, **kw):
    d = dict(dtype=1, param_dtype=2, q_heads=8, k_heads=2, dim=128, rot=128, layout=0, norm=0, eps=1e-6, amplitude=1.0)
    d.update(kw)
    return ctypes.byref(tsx.tsx_rotary_desc(*d.values()))


def test_rotary_calls(tsx, refused):
    def call(d=None, tokens=4, positions=A, wide=8, q=A, k=A, wq=None, wk=None, qo=A, ko=A, pitch=4096, head=128, **kw):
        return tsx.tsx_rotary(d or desc(tsx, **kw), tokens, positions, wide, heads(tsx, q, pitch, head),
                              heads(tsx, k, pitch, head), wq, wk, heads(tsx, qo), heads(tsx, ko), None)

    assert tsx.tsx_rotary(None, 4, A, 8, None, None, None, None, None, None, None) == tsx.TSX_ERR_INVALID
    for bad, word in ((dict(dtype=3), "dtype"), (dict(param_dtype=0), "param_dtype"), (dict(q_heads=-1), "heads"),
                      (dict(dim=0), "dim"), (dict(dim=257), "dim"), (dict(rot=127), "rot"), (dict(rot=130), "rot"),
                      (dict(layout=2), "layout"), (dict(norm=2), "norm"), (dict(eps=-1.0), "eps"),
                      (dict(amplitude=float("nan")), "amplitude"), (dict(tokens=-1), "tokens"),
                      (dict(tokens=1 << 31), "tokens"), (dict(tokens=1 << 28), "tokens"), (dict(wide=2), "bytes"),
                      (dict(wq=A), "norm"), (dict(positions=None), "positions"), (dict(q=None), "q is required"),
                      (dict(ko=None), "k_out is required"), (dict(pitch=1023), "pitches of q"),
                      (dict(head=127), "pitches of q"), (dict(pitch=-4096), "pitches of q"),
                      (dict(head=0), "pitches of q"), (dict(pitch=64), "pitches of q")):
        refused(call(**bad), tsx.TSX_ERR_INVALID, word)
    refused(call(q=A + 1), tsx.TSX_ERR_ALIGN, "q ")
    refused(call(positions=A + 4), tsx.TSX_ERR_ALIGN, "positions")
    refused(call(norm=1, wq=A + 2), tsx.TSX_ERR_ALIGN, "weight")
    assert call(tokens=0, q=None, k=None, qo=None, ko=None) == tsx.TSX_OK
    assert call(q_heads=0, k_heads=0, q=None, k=None, qo=None, ko=None) == tsx.TSX_OK
    # heads outermost are fine, as far as pitches go: the next refusal is another one
    refused(call(pitch=128, head=4 * 128, qo=None), tsx.TSX_ERR_INVALID, "q_out is required")


def test_gradient_calls(tsx, refused):
    def call(tokens=4, q=A, wq=None, gq=None, work=A, size=1 << 22, **kw):
        d = dict(norm=1)
        d.update(kw)
        x = heads(tsx, q) if q else None
        return tsx.tsx_rotary_backward(desc(tsx, **d), tokens, A, 8, heads(tsx), heads(tsx), x, x, wq, None, heads(tsx),
                                       heads(tsx), gq, None, work, size, None)

    refused(call(wq=A), tsx.TSX_ERR_INVALID, "together")
    refused(call(gq=A), tsx.TSX_ERR_INVALID, "together")
    refused(call(q=None), tsx.TSX_ERR_INVALID, "q is required")
    refused(call(norm=0), tsx.TSX_ERR_INVALID, "gradient of a norm")
    refused(call(wq=A, gq=A, work=None), tsx.TSX_ERR_INVALID, "workspace")
    refused(call(wq=A, gq=A, size=16), tsx.TSX_ERR_INVALID, "workspace")
    refused(call(wq=A, gq=A, work=A + 8), tsx.TSX_ERR_ALIGN, "workspace")
    refused(call(wq=A, gq=A + 2), tsx.TSX_ERR_ALIGN, "gradient")


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("dim,q_heads,k_heads", [(1, 1, 0), (128, 32, 8), (256, 128, 128), (256, 1, 1)])
def test_scratch_of_the_gradient(tsx, dtype, dim, q_heads, k_heads):
    """A few megabytes at most, whatever the tokens; none without a norm."""
    size = ctypes.c_size_t(99)
    for tokens in (1, 1 << 20):
        d = desc(tsx, dtype=dtype, dim=dim, rot=0, q_heads=q_heads, k_heads=k_heads, norm=1)
        assert tsx.tsx_rotary_workspace(d, tokens, ctypes.byref(size)) == tsx.TSX_OK
        assert 0 < size.value <= 4 << 20
    d = desc(tsx, dtype=dtype, dim=dim, rot=0, q_heads=q_heads, k_heads=k_heads)
    assert tsx.tsx_rotary_workspace(d, 5, ctypes.byref(size)) == tsx.TSX_OK and size.value == 0
    assert tsx.tsx_rotary_workspace(d, 5, None) == tsx.TSX_ERR_INVALID


def cache(tsx, **kw):
    c = dict(dtype=1, heads=2, dim=128, page_size=16, pages=4, page_pitch=4096, slot_pitch=256, head_pitch=128, k=A, v=A)
    c.update(kw)
    return ctypes.byref(tsx.tsx_cache(*c.values()))


def batch(tsx, **kw):
    b = dict(starts=A, lengths=A, pages=A, pages_pitch=8, seqs=3, most_pages=8)
    b.update(kw)
    return ctypes.byref(tsx.tsx_batch(*b.values()))


BAD_CACHES = [(dict(dtype=9), "dtype"), (dict(heads=0), "heads"), (dict(dim=0), "heads"), (dict(dim=257), "heads"),
              (dict(page_size=0), "slots"), (dict(page_size=1 << 21), "slots"), (dict(pages=-1), "slots"),
              (dict(page_pitch=-1), "pitch"), (dict(page_pitch=4095), "pitches"), (dict(slot_pitch=255), "pitches"),
              (dict(head_pitch=127), "pitches"), (dict(slot_pitch=0), "pitches"), (dict(k=None), "required"),
              (dict(v=None), "required")]
BAD_BATCHES = [(dict(seqs=-1), "seqs"), (dict(seqs=1 << 25), "seqs"), (dict(most_pages=-1), "most_pages"),
               (dict(pages_pitch=7), "pages_pitch"), (dict(starts=None), "required"), (dict(lengths=None), "required"),
               (dict(pages=None), "required")]


def test_append_calls(tsx, refused):
    def call(c=None, b=None, tokens=4, q=A, k=A, v=A, qo=A, **kw):
        return tsx.tsx_cache_append(desc(tsx, **kw), c or cache(tsx), b or batch(tsx), tokens, heads(tsx, q),
                                    heads(tsx, k), heads(tsx, v), None, None, heads(tsx, qo), None)

    for bad, word in BAD_CACHES:
        refused(call(c=cache(tsx, **bad)), tsx.TSX_ERR_INVALID, word)
    for bad, word in BAD_BATCHES:
        refused(call(b=batch(tsx, **bad)), tsx.TSX_ERR_INVALID, word)
    for bad in (dict(dtype=0, param_dtype=2), dict(k_heads=1), dict(dim=64, rot=64)):
        refused(call(**bad), tsx.TSX_ERR_INVALID, "cache's")
    for name in ("q", "k", "v"):
        refused(call(**{name: None}), tsx.TSX_ERR_INVALID, f"{name} is required")
    refused(call(qo=None), tsx.TSX_ERR_INVALID, "q_out is required")
    refused(call(c=cache(tsx, k=A + 1)), tsx.TSX_ERR_ALIGN, "cache")
    refused(call(b=batch(tsx, lengths=A + 2)), tsx.TSX_ERR_ALIGN, "lengths")
    assert call(tokens=0) == tsx.TSX_OK and call(b=batch(tsx, seqs=0)) == tsx.TSX_OK


def test_attention_calls(tsx, refused):
    def call(c=None, b=None, tokens=4, q_heads=8, most=1, scale=0.1, q=A, out=A, lse=None, work=A, size=1 << 27,
             pitch=4096, head=128):
        return tsx.tsx_paged_attention(c or cache(tsx), b or batch(tsx), tokens, q_heads, most, scale,
                                       heads(tsx, q, pitch, head), heads(tsx, out), lse, work, size, None)

    for bad, word in BAD_CACHES:
        refused(call(c=cache(tsx, **bad)), tsx.TSX_ERR_INVALID, word)
    for bad, word in BAD_BATCHES:
        refused(call(b=batch(tsx, **bad)), tsx.TSX_ERR_INVALID, word)
    for bad, word in ((dict(q_heads=7), "q_heads"), (dict(q_heads=0), "q_heads"), (dict(most=-1), "most_new"),
                      (dict(tokens=-1), "tokens"), (dict(tokens=1 << 29), "tokens"), (dict(scale=float("inf")), "scale"),
                      (dict(q=None), "q is required"), (dict(out=None), "out is required"), (dict(pitch=1023), "pitches"),
                      (dict(work=None), "workspace"), (dict(size=1000), "workspace")):
        refused(call(**bad), tsx.TSX_ERR_INVALID, word)
    refused(call(c=cache(tsx, dtype=2)), tsx.TSX_ERR_UNSUPPORTED, "fp32")
    refused(call(c=cache(tsx, dim=124)), tsx.TSX_ERR_UNSUPPORTED, "multiple of 8")
    for bad in (dict(q=A + 2), dict(out=A + 8), dict(pitch=4100), dict(head=132), dict(c=cache(tsx, k=A + 8)),
                dict(c=cache(tsx, page_pitch=4100)), dict(lse=A + 2), dict(work=A + 8)):
        refused(call(**bad), tsx.TSX_ERR_ALIGN, "")
    assert call(tokens=0, q=None, out=None) == tsx.TSX_OK and call(b=batch(tsx, seqs=0)) == tsx.TSX_OK


@pytest.mark.parametrize("dim", [8, 64, 80, 128, 256])
@pytest.mark.parametrize("most", [0, 1, 2, 1 << 20])
def test_scratch_of_attention(tsx, dim, most):
    """The header's 64 MB hold, and tokens do not matter."""
    c = cache(tsx, dim=dim, slot_pitch=512, head_pitch=256, page_pitch=1 << 20)
    sizes = []
    for tokens in (1, 1 << 16):
        size = ctypes.c_size_t(99)
        assert tsx.tsx_paged_attention_workspace(c, tokens, 8, most, ctypes.byref(size)) == tsx.TSX_OK
        sizes.append(size.value)
    assert sizes[0] == sizes[1] and 0 < sizes[0] <= 64 << 20 and sizes[0] % 16 == 0


# ------------------------------------------------- the plain definitions


def test_definitions_against_differences():
    rng = np.random.default_rng(0)
    x, w, d = rng.standard_normal((3, 2, 12)), rng.standard_normal(12), rng.standard_normal((3, 2, 12))
    f, amp = ref.frequencies(8, scaling=("yarn", 4.0, 64))
    pos = np.array([0, 5, 1000])
    for layout in ("half", "interleaved"):
        def y(x, w):
            return ref.turn(ref.norm(x, w, 1e-3)[0], pos, f, amp, layout)

        dx, dw = ref.norm_backward(ref.turn(d, pos, f, amp, layout, back=True), x, w, 1e-3)
        t = 1e-6
        for at in np.ndindex(x.shape):
            u = np.zeros_like(x)
            u[at] = t
            assert abs(((y(x + u, w) - y(x - u, w)) * d).sum() / (2 * t) - dx[at]) < 1e-7
        for c in range(12):
            u = np.zeros(12)
            u[c] = t
            assert abs(((y(x, w + u) - y(x, w - u)) * d).sum() / (2 * t) - dw[c]) < 1e-7
        # a rotation keeps a pair's length, up to the amplitude
        a, b = ref.pairs(8, layout)
        z = ref.turn(x, pos, f, amp, layout)
        np.testing.assert_allclose(z[..., a]**2 + z[..., b]**2, amp**2 * (x[..., a]**2 + x[..., b]**2))


def test_attention_definition_is_a_softmax():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 3, 4, 1, 8))
    q = rng.standard_normal((2, 2, 8))
    out, lse = ref.attend(q, k, v, np.array([0, 2]), np.array([7]), np.array([[2, 0]]), 0.3)
    keys, values = (np.concatenate([t[2], t[0]])[:, 0] for t in (k, v))
    for t, n in ((0, 6), (1, 7)):
        x = q[t] @ keys[:n].T * 0.3
        w = np.exp(x) / np.exp(x).sum(-1, keepdims=True)
        np.testing.assert_allclose(out[t], w @ values[:n])
        np.testing.assert_allclose(lse[t], np.log(np.exp(x).sum(-1)))


def test_caches_and_batches_of_other_shapes_are_refused(tsx):
    """By the class, before any call: host tensors stand for a device's."""
    import torch

    att = tsx.PagedAttention("bf16", 4, 2, 64, 16)
    good = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    dev = good.get_device()
    assert att._cache((good, good), dev).pages == 3
    assert att._cache((good.transpose(1, 2).contiguous().transpose(1, 2),) * 2, dev).head_pitch == 16 * 64
    for k, v, word in ((good.half(), good.half(), "bf16"), (good, good.half(), "bf16"), (good[0], good[0], "shape"),
                       (good[:, :8], good[:, :8], "shape"), (good[:, :, :1], good[:, :, :1], "shape"),
                       (good[..., :32], good[..., :32], "shape"), (good, good[:2], "shape"),
                       (good, torch.zeros(3, 16, 2, 128, dtype=good.dtype)[..., :64], "strides"),
                       (torch.zeros(3, 16, 2, 128, dtype=good.dtype)[..., ::2],) * 2 + ("strides",)):
        with pytest.raises(tsx.TsxError, match=word):
            att._cache((k, v), dev)
    i32 = torch.zeros(9, dtype=torch.int32)
    pages = torch.zeros(3, 5, dtype=torch.int32)
    assert att._batch(tsx.Batch(i32[:4], i32[:3], pages, 1), dev).most_pages == 5
    assert att._batch(tsx.Batch(i32[:4], i32[:3], torch.zeros(3, 9, dtype=torch.int32)[:, :5], 1), dev).pages_pitch == 9
    for b, word in ((tsx.Batch(i32[:4].long(), i32[:3], pages, 1), "int32"), (tsx.Batch(i32[:3], i32[:3], pages, 1), "seqs"),
                    (tsx.Batch(i32[:4], i32[:4], pages, 1), "seqs"), (tsx.Batch(i32[:4], i32[:3], pages[0], 1), "seqs"),
                    (tsx.Batch(i32[:4], pages[:, :1], pages, 1), "seqs"), (tsx.Batch(i32[:8:2], i32[:3], pages, 1), "contig"),
                    (tsx.Batch(i32[:4], i32[:6:2], pages, 1), "contig"),
                    (tsx.Batch(i32[:4], i32[:3], torch.zeros(3, 10, dtype=torch.int32)[:, ::2], 1), "contig")):
        with pytest.raises(tsx.TsxError, match=word):
            att._batch(b, dev)
