"""Workloads of the training operators: channels-last group norm with an
activation, gated activations, and activation checkpoints held in 8 bits.

``listed()`` names the workloads, ``prepare`` makes one's inputs, ``run`` does
one pass: with elementary torch operations in 32 bits, or (``own``) through
the library.  ``exact`` gives the same outputs from the definitions in 64 bits
and ``work`` the bytes and operations that a pass cannot do without.

The operators, for x of [n, l, c] in g groups of c / g channels:

  group norm   xhat = (x - mean) / sqrt(var + eps) over the l rows and the
               channels of a group; y = act(xhat * weight + bias)
  gated act    h = act(gate) * up, element by element
  checkpoint   each run of `block` channels of a row is held as 8-bit numbers
               q and one fp32 scale: amax / 127 and whole numbers for int8,
               amax / 448 and e4m3 numbers for e4m3.  A block whose largest
               magnitude is under 2^-119 is held as zeros.

act is none, silu (z sigmoid(z)) or gelu (its tanh form).  A backward pass
from a checkpoint is the same formula with q * scale in the place of the saved
tensor; the statistics are those of the forward pass.
"""

from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
TOP = {"int8": 127.0, "e4m3": 448.0}
TINY = 2.0 ** -119


def listed():
    return [
        # group norm over each head's output, one decoding step of 16 sequences
        dict(name="norm token", op="norm", dtype="bf16", n=16, l=1, c=4096, g=32, act="none", extra=0),
        # the same over a prompt of 8192 tokens
        dict(name="norm prompt", op="norm", dtype="bf16", n=8192, l=1, c=4096, g=32, act="none", extra=0),
        # feature maps of 64 x 64 positions in half precision, ten channels to a group
        dict(name="norm feature maps", op="norm", dtype="f16", n=8, l=4096, c=320, g=32, act="silu", extra=0),
        # one image of 512 x 512 positions, four channels to a group
        dict(name="norm image", op="norm", dtype="bf16", n=1, l=262144, c=128, g=32, act="silu", extra=0),
        # gradient in a deep stage of such a network; x is a slice of a wider tensor
        dict(name="norm gradient", op="norm_grad", dtype="bf16", n=4, l=1024, c=1280, g=32, act="silu", extra=640),
        # gradient with nothing round about its sizes, in single precision
        dict(name="norm gradient odd", op="norm_grad", dtype="f32", n=3, l=1009, c=198, g=11, act="gelu", extra=0),
        # a training step of one layer that keeps its input in 8 bits: forward, then backward from the checkpoint
        dict(name="norm step int8", op="norm_step", dtype="bf16", n=4, l=16384, c=512, g=32, act="silu", extra=0,
             form="int8", block=128),
        # 64 tokens' activations to 8 bits and back
        dict(name="checkpoint small", op="pack", dtype="bf16", rows=64, cols=4096, form="int8", block=128),
        # a batch's activations, the size of this library's bf16 benchmark
        dict(name="checkpoint large", op="pack", dtype="bf16", rows=16384, cols=16384, form="int8", block=128),
        # a gated feed-forward's activation, both passes, for a micro-batch of 32 tokens
        dict(name="gated step small", op="gated_step", dtype="bf16", rows=32, cols=8192, act="silu", form="int8",
             block=128),
        # its backward pass for 16384 tokens from e4m3 checkpoints, h recomputed for the next layer's weight gradient
        dict(name="gated gradient large", op="gated_grad", dtype="bf16", rows=16384, cols=12288, act="silu",
             form="e4m3", block=64),
        # forward in single precision with rows of odd length, gate and up side by side in one tensor
        dict(name="gated ragged", op="gated", dtype="f32", rows=1777, cols=2731, act="gelu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "norm_step", "pack", "gated", "gated_grad", "gated_step"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op.startswith("norm"):
        case["act"] = rng.choice(["none", "silu", "silu", "gelu"])
        g = rng.choice([1, 2, 4, 8, 16, 32, 32, 32, 5, 11])
        per = rng.choice([1, 2, 4, 8, 10, 16, 20, 40, 64, 128]) if rng.random() < 0.7 else _log(rng, 1, 256)
        c = g * per
        total = _log(rng, 1 << 15, 1 << 25)
        l = min(_log(rng, 1, 65536), max(1, total // c))
        if rng.random() < 0.2:
            l = 1
        case.update(n=min(16384, max(1, total // (l * c))), l=l, c=c, g=g,
                    extra=rng.choice([0, 0, 0, 8, 24, c]) if op != "norm_step" else 0)
    else:
        total = _log(rng, 1 << 13, 1 << 26)
        cols = rng.choice([128, 256, 768, 1024, 2048, 4096, 5120, 8192, 11008]) if rng.random() < 0.6 \
            else _log(rng, 16, 16384)
        case.update(rows=max(1, min(65536, total // cols)), cols=cols)
        if op != "pack":
            case["act"] = rng.choice(["silu", "gelu"])
    if op in ("norm_step", "pack", "gated_grad", "gated_step"):
        case.update(form=rng.choice(["int8", "int8", "e4m3"]), block=rng.choice([128, 128, 64, 32]))
    return case


# ---------------------------------------------------------------- inputs


def _activations(gen, shape, dtype, extra=0):
    """Values as activations have them: every channel with its own spread and
    offset, a few channels far larger than the rest; `extra` channels more in
    a row than the tensor that is returned shows."""
    c = shape[-1]
    wide = (*shape[:-1], c + extra)
    x = torch.randn(wide, generator=gen, device="cuda")
    spread = torch.exp(0.5 * torch.randn(c + extra, generator=gen, device="cuda"))
    spread = torch.where(torch.rand(c + extra, generator=gen, device="cuda") < 0.01, 8 * spread, spread)
    x.mul_(spread).add_(0.5 * torch.randn(c + extra, generator=gen, device="cuda"))
    return x.to(TORCH[dtype])[..., :c]


def _gradient(gen, shape, dtype):
    return (0.1 * torch.randn(shape, generator=gen, device="cuda")).to(TORCH[dtype])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case)
    op, dt = case["op"], case["dtype"]
    if op.startswith("norm"):
        n, l, c = case["n"], case["l"], case["c"]
        s["x"] = _activations(gen, (n, l, c), dt, case["extra"])
        s["weight"] = 1 + 0.2 * torch.randn(c, generator=gen, device="cuda")
        s["bias"] = 0.2 * torch.randn(c, generator=gen, device="cuda")
        if op != "norm":
            s["dy"] = _gradient(gen, (n, l, c), dt)
        if op == "norm_grad":
            s["mean"], s["rstd"] = _statistics(s["x"].float(), case["g"])
    elif op == "pack":
        s["x"] = _activations(gen, (case["rows"], case["cols"]), dt)
    else:
        rows, cols = case["rows"], case["cols"]
        if op == "gated_grad":   # what a forward pass left
            s["gate"] = _quantise(_activations(gen, (rows, cols), dt).float(), case["form"], case["block"])
            s["up"] = _quantise(_activations(gen, (rows, cols), dt).float(), case["form"], case["block"])
        else:   # one projection gives both, side by side
            both = torch.cat([_activations(gen, (rows, cols), dt), _activations(gen, (rows, cols), dt)], 1)
            s["gate"], s["up"] = both[:, :cols], both[:, cols:]
        if op != "gated":
            s["dh"] = _gradient(gen, (rows, cols), dt)
    if own:   # the operator's handle, which a program makes once for its shape
        import pipelined_elementwise_streaming_gb300 as tsx

        if op.startswith("norm"):
            s["handle"] = tsx.GroupNorm(dt, n, l, c, case["g"], act=case["act"], eps=EPS,
                                        x_pitch=c + case["extra"], form=case.get("form", "int8"),
                                        block=case.get("block", 128))
        elif op == "pack":
            s["handle"] = tsx.Packer(dt, case["rows"], case["cols"], form=case["form"], block=case["block"])
        else:
            s["handle"] = tsx.GatedAct(dt, rows, cols, act=case["act"],
                                       in_pitch=cols if op == "gated_grad" else 2 * cols,
                                       form=case.get("form", "int8"), block=case.get("block", 128))
    return s


# ------------------------------------------------------------- plain form


def _statistics(x, g):
    n, l, c = x.shape
    v = x.reshape(n, l, g, c // g)
    mean = v.mean((1, 3), keepdim=True)
    var = (v - mean).square().mean((1, 3))
    return mean.reshape(n, g), 1 / torch.sqrt(var + EPS)


def _per_channel(v, c):
    """[n, g] -> [n, 1, c]"""
    n, g = v.shape
    return v.reshape(n, 1, g, 1).expand(n, 1, g, c // g).reshape(n, 1, c)


def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _norm(x, weight, bias, g, act):
    x = x.float()
    mean, rstd = _statistics(x, g)
    c = x.shape[-1]
    z = (x - _per_channel(mean, c)) * _per_channel(rstd, c) * weight + bias
    return _act(z, act), mean, rstd


def _norm_backward(dy, x, weight, bias, mean, rstd, g, act):
    n, l, c = x.shape
    r = _per_channel(rstd, c)
    xhat = (x - _per_channel(mean, c)) * r
    dz = dy.float() * _act_slope(xhat * weight + bias, act)
    dweight, dbias = (dz * xhat).sum((0, 1)), dz.sum((0, 1))
    d = dz * weight
    m1 = d.reshape(n, l, g, c // g).mean((1, 3))
    m2 = (d * xhat).reshape(n, l, g, c // g).mean((1, 3))
    return r * (d - _per_channel(m1, c) - xhat * _per_channel(m2, c)), dweight, dbias


def _quantise(x, form, block):
    """(q as int8 or e4m3 of x's shape [rows, cols], fp32 scales [rows, blocks])"""
    rows, cols = x.shape
    blocks = -(-cols // block)
    v = torch.nn.functional.pad(x, (0, blocks * block - cols)).reshape(rows, blocks, block)
    amax = v.abs().amax(-1)
    scale = torch.where(amax < TINY, torch.zeros_like(amax), amax * (1 / TOP[form]))
    inv = torch.where(scale > 0, 1 / scale, scale)
    v = v * inv[..., None]
    q = torch.round(v).to(torch.int8) if form == "int8" else v.to(torch.float8_e4m3fn)
    return q.reshape(rows, blocks * block)[:, :cols].contiguous(), scale


def _values(q, scale, block):
    return q.float() * scale.repeat_interleave(block, 1)[:, : q.shape[1]]


def _plain(s):
    case = s["case"]
    op, t = case["op"], TORCH[case["dtype"]]
    if op == "norm":
        y, mean, rstd = _norm(s["x"], s["weight"], s["bias"], case["g"], case["act"])
        return y.to(t), mean, rstd
    if op == "norm_grad":
        dx, dw, db = _norm_backward(s["dy"], s["x"].float(), s["weight"], s["bias"], s["mean"], s["rstd"], case["g"],
                                    case["act"])
        return dx.to(t), dw, db
    if op == "norm_step":
        x = s["x"]
        y, mean, rstd = _norm(x, s["weight"], s["bias"], case["g"], case["act"])
        saved = _values(*_quantise(x.reshape(-1, x.shape[-1]).float(), case["form"], case["block"]), case["block"])
        dx, dw, db = _norm_backward(s["dy"], saved.reshape(x.shape), s["weight"], s["bias"], mean, rstd, case["g"],
                                    case["act"])
        return y.to(t), mean, rstd, dx.to(t), dw, db
    if op == "pack":
        q, scale = _quantise(s["x"].float(), case["form"], case["block"])
        return _values(q, scale, case["block"]).to(t), scale
    if op == "gated":
        return (_act(s["gate"].float(), case["act"]) * s["up"].float()).to(t)
    h = None
    gate, up = s["gate"], s["up"]
    if op == "gated_step":
        h = (_act(gate.float(), case["act"]) * up.float()).to(t)
        gate, up = (_quantise(v.float(), case["form"], case["block"]) for v in (gate, up))
    a, b = _values(*gate, case["block"]), _values(*up, case["block"])
    dh = s["dh"].float()
    dgate, dup = (dh * b * _act_slope(a, case["act"])).to(t), (dh * _act(a, case["act"])).to(t)
    if op == "gated_grad":
        h = (_act(a, case["act"]) * b).to(t)
    return h, dgate, dup


# -------------------------------------------------------------- the library


def _library(s):
    op, f = s["case"]["op"], s["handle"]
    if op == "norm":
        return f.forward(s["x"], s["weight"], s["bias"])
    if op == "norm_grad":
        return f.backward(s["dy"], s["x"], s["weight"], s["bias"], s["mean"], s["rstd"])
    if op == "norm_step":
        y, mean, rstd, saved = f.forward(s["x"], s["weight"], s["bias"], checkpoint=True)
        return (y, mean, rstd, *f.backward(s["dy"], saved, s["weight"], s["bias"], mean, rstd))
    if op == "pack":
        saved = f.pack(s["x"])
        return f.unpack(saved), saved.scale
    if op == "gated":
        return f.forward(s["gate"], s["up"])
    if op == "gated_step":
        h, gate, up = f.forward(s["gate"], s["up"], checkpoint=True)
        return (h, *f.backward(s["dh"], gate, up))
    dgate, dup, h = f.backward(s["dh"], s["gate"], s["up"], recompute=True)
    return h, dgate, dup


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------ what it needs


def work(case):
    """Each input read once, each output (a checkpoint too) written once."""
    op, es = case["op"], SIZE[case["dtype"]]
    if op.startswith("norm"):
        e, c, stats = case["n"] * case["l"] * case["c"], case["c"], 8 * case["n"] * case["g"]
        fwd, bwd = 2 * es * e + 8 * c + stats, 3 * es * e + 16 * c + stats
        if op == "norm":
            return {"bytes": fwd, "flops": 12 * e}
        if op == "norm_grad":
            return {"bytes": bwd, "flops": 24 * e}
        held = e + 4 * case["n"] * case["l"] * -(-c // case["block"])
        return {"bytes": fwd + bwd - es * e + 2 * held, "flops": 40 * e}
    e = case["rows"] * case["cols"]
    if op == "gated":
        return {"bytes": 3 * es * e, "flops": 8 * e}
    held = e + 4 * case["rows"] * -(-case["cols"] // case["block"])
    if op == "pack":
        return {"bytes": 2 * es * e + 2 * held, "flops": 5 * e}
    if op == "gated_grad":
        return {"bytes": 4 * es * e + 2 * held, "flops": 18 * e}
    return {"bytes": 6 * es * e + 4 * held, "flops": 32 * e}


# --------------------------------------------------------- 64-bit definition


def _sigmoid64(z):
    return torch.special.expit(z)


def _act64(z, act):
    """(act(z), act'(z)) from the sigmoid: tanh(u) = 2 sigmoid(2 u) - 1."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "silu":
        p = _sigmoid64(z)
        return z * p, p + z * p * _sigmoid64(-z)
    k = 2 * math.sqrt(2 / math.pi)
    u = k * z * (1 + 0.044715 * z ** 2)
    p = _sigmoid64(u)
    return z * p, p + z * p * _sigmoid64(-u) * k * (1 + 0.134145 * z ** 2)


def _held64(x, form, block):
    """What a checkpoint of x [rows, cols] stands for, and its scales."""
    x = x.double()
    out, scales = torch.empty_like(x), []
    for at in range(0, x.shape[1], block):
        b = x[:, at:at + block]
        top = b.abs().max(1, keepdim=True).values
        top = torch.where(top < TINY, torch.zeros_like(top), top)
        step = top / TOP[form]
        v = torch.where(step > 0, b / torch.where(step > 0, step, torch.ones_like(step)), torch.zeros_like(b))
        if form == "e4m3":   # three bits of mantissa, the smallest normal number 2^-6
            unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
            v = torch.round(v / unit) * unit
        else:
            v = torch.round(v)
        out[:, at:at + block] = v * step
        scales.append(step)
    return out, torch.cat(scales, 1)


def _norm64(x, w, b, g, act, saved=None, dy=None):
    """[y, mean, rstd] and, with dy, [dx, dweight, dbias] from `saved`."""
    n, l, c = x.shape
    x4 = x.double().view(n, l, g, c // g)
    m = l * (c // g)
    mean = torch.einsum("nlgk->ng", x4) / m
    var = torch.einsum("nlgk,nlgk->ng", x4, x4) / m - mean ** 2
    rstd = (var + EPS) ** -0.5
    w4, b4 = w.double().view(g, c // g), b.double().view(g, c // g)
    hat = (x4 - mean[:, None, :, None]) * rstd[:, None, :, None]
    out = [_act64(hat * w4 + b4, act)[0].view(n, l, c), mean, rstd]
    if dy is None:
        return out, []
    hat = (saved.double().view(n, l, g, c // g) - mean[:, None, :, None]) * rstd[:, None, :, None]
    dz = dy.double().view(n, l, g, c // g) * _act64(hat * w4 + b4, act)[1]
    p, q = torch.einsum("nlgk->ngk", dz), torch.einsum("nlgk,nlgk->ngk", dz, hat)
    s1, s2 = (torch.einsum("ngk,gk->ng", v, w4)[:, None, :, None] / m for v in (p, q))
    dx = (dz * w4 - s1 - hat * s2) * rstd[:, None, :, None]
    return out, [dx.view(n, l, c), q.sum(0).view(c), p.sum(0).view(c)]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        x, dy = s["x"].contiguous(), s.get("dy")
        args = (x, s["weight"], s["bias"], case["g"], case["act"])
        if op == "norm":
            return tuple(_norm64(*args)[0])
        if op == "norm_grad":
            return tuple(_norm64(*args, x, dy)[1])
        held = _held64(x.view(-1, x.shape[-1]), case["form"], case["block"])[0].view(x.shape)
        out, grads = _norm64(*args, held, dy)
        return (*out, *grads)
    if op == "pack":
        return _held64(s["x"], case["form"], case["block"])
    if op == "gated":
        return _act64(s["gate"].double(), case["act"])[0] * s["up"].double()
    if op == "gated_step":
        h = _act64(s["gate"].double(), case["act"])[0] * s["up"].double()
        a, b = (_held64(s[k], case["form"], case["block"])[0] for k in ("gate", "up"))
    else:
        a, b = (_stands_for64(*s[k], case["block"]) for k in ("gate", "up"))
        h = _act64(a, case["act"])[0] * b
    value, slope = _act64(a, case["act"])
    dh = s["dh"].double()
    return h, dh * b * slope, dh * value


def _stands_for64(q, scale, block):
    out = q.double()
    for k in range(scale.shape[1]):
        out[:, k * block:(k + 1) * block] *= scale[:, k:k + 1].double()
    return out
