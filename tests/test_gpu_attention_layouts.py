"""The operators around attention on a GPU: outputs in the place of inputs, calls
of very many tokens, caches that are part of something wider, first calls in a
capture, and several threads at once."""

import threading

import pytest

from tests import _gpu
from tests._gpu import torch
from tests.test_gpu_attend import made
from tests.test_gpu_cache import int32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


def tensors(dtype, dim, tokens=300, hq=5, hk=2):
    gen = torch.Generator(device="cuda").manual_seed(dim)
    return [torch.randn(tokens, h, dim, generator=gen, device="cuda").to(_gpu.TORCH_DTYPE[dtype])
            for h in (hq, hk, hq, hk)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,rot", [(128, 64), (50, 20)])
@pytest.mark.parametrize("over", ["gradient", "input"])
def test_gradients_in_place(tsx, dtype, dim, rot, over):
    """Over the gradients that come in, or over the inputs that were kept."""
    q, k, dq, dk = tensors(dtype, dim)
    w = [torch.rand(dim, device="cuda") + 0.5 for _ in range(2)]
    pos = torch.arange(300, device="cuda")
    for layout in ("half", "interleaved"):
        f = tsx.Rotary(dtype, 5, 2, dim, rot=rot, layout=layout, norm="rms")
        want = f.backward(dq, dk, pos, q, k, *w)
        a, b, c, d = (t.clone() for t in (q, k, dq, dk))
        out = (c, d) if over == "gradient" else (a, b)
        got = f.backward(c, d, pos, a, b, *w, q_out=out[0], k_out=out[1])
        assert got[0] is out[0] and got[1] is out[1]
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        plain = tsx.Rotary(dtype, 5, 2, dim, rot=rot, layout=layout)
        want = plain.backward(dq, dk, pos)
        got = plain.backward(c.copy_(dq), d.copy_(dk), pos, q_out=c, k_out=d)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("dtype,dim,heads", [("bf16", 8, 1), ("f16", 128, 3), ("f32", 20, 2)])
def test_very_many_tokens(tsx, dtype, dim, heads):
    """A call of 300001 tokens gives each token what a call of a few gives it."""
    n = 300001
    f = tsx.Rotary(dtype, heads, 0, dim, norm="rms")
    x = torch.randn(n, heads, dim, device="cuda").to(_gpu.TORCH_DTYPE[dtype])
    w = torch.rand(dim, device="cuda")
    pos = torch.randint(1 << 40, (n,), device="cuda")
    y, _ = f.forward(x, None, pos, w)
    d, _, dw, _ = f.backward(y, None, pos, x, None, w)
    at = [slice(0, 7), slice(150000, 150033), slice(n - 5, n)]
    for s in at:
        a, _ = f.forward(x[s], None, pos[s].contiguous(), w)
        b, *_ = f.backward(y[s], None, pos[s].contiguous(), x[s], None, w)
        assert torch.equal(y[s], a) and torch.equal(d[s], b)
    assert torch.isfinite(dw).all()


@pytest.mark.parametrize("dim,page", [(128, 16), (64, 24)])
def test_keys_and_values_in_one_tensor(tsx, dim, page):
    """Pages of keys and values by turns, heads before slots, in a tensor with more
    around them; queries turned in place."""
    att, q, cache, batch = made(tsx, "bf16", 4, 2, dim, page, [20, 1], [130, 40])
    pages = cache[0].shape[0]
    wide = torch.full((pages, 2, 3, page, dim + 8), 7.0, dtype=q.dtype, device="cuda")
    part = tuple(wide[:, i, :2, :, :dim].transpose(1, 2) for i in range(2))
    for p, c in zip(part, cache):
        p.copy_(c)
    rope = tsx.Rotary("bf16", 4, 2, dim)
    turned = tsx.PagedAttention("bf16", 4, 2, dim, page, rotary=rope)
    k, v = (torch.randn(21, 2, dim, device="cuda").bfloat16() for _ in range(2))
    mine = q.clone()
    a = turned.append(q, k, v, cache, batch)
    b = turned.append(mine, k, v, part, batch, out=mine)
    assert b is mine and torch.equal(a, b)
    bits = torch.int16
    assert all(torch.equal(p.contiguous().view(bits), c.contiguous().view(bits)) for p, c in zip(part, cache))
    for most in (1, 100):
        held = batch._replace(most_new=most)
        assert torch.equal(turned.forward(a, cache, held), turned.forward(a, part, held))
    wide[:, :, :2, :, :dim] = 7
    assert (wide == 7).all()


def test_first_calls_within_a_capture(tsx):
    """Shapes that no call has had before, captured at once."""
    att, q, cache, batch = made(tsx, "f16", 3, 1, 40, 16, [9, 1], [33, 70])
    wide, q2, cache2, batch2 = made(tsx, "f16", 2, 1, 200, 16, [2], [90])
    f = tsx.Rotary("f16", 3, 1, 40, norm="rms")
    pos, w = torch.arange(10, device="cuda"), torch.ones(40, device="cuda")
    k = q[:, :1].contiguous()
    torch.cuda.synchronize()

    def run():
        return (att.forward(q, cache, batch), wide.forward(q2, cache2, batch2),
                *f.backward(*f.forward(q, k, pos, w, w), pos, q, k, w, w))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, run()))


def test_several_threads(tsx):
    """One handle, several threads with streams of their own."""
    att, q, cache, batch = made(tsx, "bf16", 8, 2, 128, 16, [60, 1, 1], [300, 50, 900])
    f = tsx.Rotary("bf16", 8, 2, 128, norm="rms")
    pos, w = torch.arange(62, device="cuda"), torch.ones(128, device="cuda")
    k = q[:, :2].contiguous()
    want = (att.forward(q, cache, batch), *f.forward(q, k, pos, w, w))
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(30):
            got = (att.forward(q, cache, batch, stream=s), *f.forward(q, k, pos, w, w, stream=s))
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want)):
                bad.append(1)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_refusals_leave_the_next_call_alone(tsx):
    """A refused call writes nothing and is not in the way of the next."""
    att = tsx.PagedAttention("f32", 2, 1, 64, 16)
    cache = att.new_cache(2)
    batch = tsx.Batch(int32([0, 1]), int32([1]), int32([[0]]), 1)
    q = torch.ones(1, 2, 64, device="cuda")
    k = torch.ones(1, 1, 64, device="cuda")
    out = torch.full_like(q, 9)
    with pytest.raises(tsx.TsxError) as e:
        att.forward(q, cache, batch, out=out)
    assert e.value.code == tsx.TSX_ERR_UNSUPPORTED and (out == 9).all()
    half = tsx.PagedAttention("bf16", 2, 1, 64, 16)
    with pytest.raises(tsx.TsxError) as e:   # queries that start off 16 bytes
        half.forward(torch.ones(1, 2, 65, device="cuda").bfloat16()[..., 1:], half.new_cache(2), batch)
    assert e.value.code == tsx.TSX_ERR_ALIGN
    assert torch.equal(att.append(q, k, k, cache, batch), q) and (cache[0][0, 0] == 1).all()
