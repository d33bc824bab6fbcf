"""Workloads of the operators around attention: rotary positions, norms of
queries and keys with the rotation in the same pass, appending to a paged
cache of keys and values, and attention of new tokens over such a cache.

``listed()`` names the workloads, ``prepare`` makes one's inputs, ``run`` does
one pass: with elementary torch operations in 32 bits (angles in 64), or
(``own``) through the library.  ``exact`` gives the same outputs from the
definitions in 64 bits and ``work`` the bytes and operations that a pass cannot
do without.

The operators, for queries [tokens, heads, dim], keys and values [tokens,
kv_heads, dim], which a projection leaves side by side in one tensor:

  rotary    the first `rot` channels of a head are pairs, channel i with
            i + rot / 2 ("half") or 2 i with 2 i + 1 ("interleaved"); pair i of
            a token at position p turns by the angle p f[i] and grows by the
            factor `amplitude`
  norm      x rstd weight before the rotation, rstd = 1 / sqrt(mean of x^2 over
            the head + eps), one weight for the queries and one for the keys
  append    queries and keys normed and rotated; keys and values go to the
            sequences' pages, queries to a tensor of their own
  attend    softmax(scale q k^T) v over the keys up to each token's own place

Frequencies: f[i] = base^(-2 i / rot), for long contexts scaled "linear" (all
divided by a factor), "ntk" (a larger base) or "yarn" (slow ones divided, fast
ones kept, a ramp between, and an amplitude).
"""

from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # one decoding step of 8 sequences far into a context stretched to 16 times its length
        dict(name="rotary token", op="rotary", dtype="bf16", tokens=8, hq=32, hk=8, dim=128, rot=128, layout="half",
             scaling="yarn", far=524288),
        # a prompt of odd length, two thirds of each head turned, neighbouring channels as pairs
        dict(name="rotary prompt", op="rotary", dtype="f16", tokens=8191, hq=16, hk=16, dim=96, rot=64,
             layout="interleaved", scaling="linear", far=8191),
        # both passes of a training step in single precision
        dict(name="rotary step", op="rotary_step", dtype="f32", tokens=4096, hq=12, hk=12, dim=64, rot=64,
             layout="half", scaling="none", far=4096),
        # heads normed and turned in one decoding step of 32 sequences
        dict(name="norm token", op="norm", dtype="bf16", tokens=32, hq=32, hk=4, dim=128, rot=128, layout="half",
             scaling="none", far=32768),
        # both passes for a micro-batch of 8192 tokens, gradients of both weights among the outputs
        dict(name="norm step", op="norm_step", dtype="bf16", tokens=8192, hq=32, hk=8, dim=128, rot=128,
             layout="half", scaling="none", far=4096),
        # a gradient with nothing round about its sizes: heads of 72 channels, 40 of them turned
        dict(name="norm gradient odd", op="norm_grad", dtype="f16", tokens=1009, hq=6, hk=2, dim=72, rot=40,
             layout="interleaved", scaling="none", far=1009),
        # one token to each of 48 sequences of up to 2048, pages of 16
        dict(name="append token", op="append", dtype="bf16", seqs=48, new=1, longest=2048, hq=32, hk=8, dim=128,
             rot=128, layout="half", scaling="none", page=16, norm=True),
        # chunks of a ragged batch of prompts, pages of 64, keys turned and not normed
        dict(name="append chunk", op="append", dtype="f16", seqs=7, new=1500, longest=4096, hq=16, hk=8, dim=64,
             rot=64, layout="half", scaling="ntk", page=64, norm=False),
        # one decoding step of 64 sequences of 1000 to 16000 tokens
        dict(name="attend tokens", op="attend", dtype="bf16", seqs=64, new=1, longest=16384, hq=32, hk=8, dim=128,
             page=16),
        # one decoding step of a single long document
        dict(name="attend long", op="attend", dtype="f16", seqs=1, new=1, longest=100003, hq=16, hk=2, dim=64,
             page=64),
        # chunks of 1024 tokens of two prompts
        dict(name="attend chunk", op="attend", dtype="bf16", seqs=2, new=1024, longest=16384, hq=32, hk=8, dim=128,
             page=32),
        # a ragged batch, some sequences with one new token and some with hundreds, five queries to a key
        dict(name="attend ragged", op="attend", dtype="f16", seqs=12, new=300, longest=3000, hq=10, hk=2, dim=64,
             page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_step", "norm", "norm_step", "norm_grad", "append", "append", "attend",
                     "attend", "attend"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16"]))
    hk = rng.choice([1, 2, 4, 8, 3])
    dim = rng.choice([64, 128, 128, 128, 96, 80])
    case.update(hk=hk, hq=hk * rng.choice([1, 2, 4, 4, 5, 8]), dim=dim)
    if op != "attend":
        if rng.random() < 0.25:
            case["dtype"] = "f32"
        case.update(layout=rng.choice(["half", "half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    rot=dim if rng.random() < 0.6 else 2 * rng.randint(4, dim // 2))
    if op in ("append", "attend"):
        case["page"] = rng.choice([16, 16, 32, 64, 128, 24])
        if op == "append":
            case.update(seqs=_log(rng, 1, 64), new=1 if rng.random() < 0.4 else _log(rng, 2, 1500),
                        norm=rng.random() < 0.5)
            case["longest"] = max(case["new"], _log(rng, 64, min(4096, 120000 // case["seqs"])))
        elif rng.random() < 0.5:   # single tokens
            seqs = _log(rng, 1, 128)
            case.update(seqs=seqs, new=1, longest=_log(rng, 64, min(131072, 262144 // seqs)))
        else:
            seqs = _log(rng, 1, 16)
            new = _log(rng, 2, 2048 // seqs)
            case.update(seqs=seqs, new=new, longest=max(new, _log(rng, 64, 16384)))
    else:
        tokens = _log(rng, 1, min(16384, (1 << 25) // ((case["hq"] + hk) * dim)))
        case.update(tokens=tokens, far=max(1, _log(rng, 16, 1 << 20)))
    return case


# ---------------------------------------------------------------- inputs


def _projection(gen, tokens, heads, dim, dtype):
    """What a projection leaves: every head with its own size, a few channels
    far larger than the rest."""
    size = torch.exp(0.4 * torch.randn(heads, dim, generator=gen, device="cuda"))
    size = torch.where(torch.rand(heads, dim, generator=gen, device="cuda") < 0.01, 6 * size, size)
    return (torch.randn(tokens, heads, dim, generator=gen, device="cuda") * size).to(TORCH[dtype])


def _scaling(case):
    return {"none": None, "linear": ("linear", 4.0), "ntk": ("ntk", 4.0), "yarn": ("yarn", 16.0, 32768)}[
        case["scaling"]]


def _lengths(case):
    """Ragged sequences: how many tokens of each are new, and how long it is
    with them.  The first has the most of both, every third a single new one;
    the lengths are spread over their logarithm."""
    seqs, new, longest = case["seqs"], case["new"], case["longest"]
    least = max(1, longest // 16)
    count, length = [new], [longest]
    for k in range(1, seqs):
        u, v = k * 0.6180339887 % 1, k * 0.7548776662 % 1
        count.append(1 if new == 1 or k % 3 == 2 else max(1, int(new * (0.3 + 0.7 * u))))
        length.append(max(count[k], int(least * (longest / least) ** v)))
    return count, length


def _batch(case, gen):
    """The sequences of `_lengths` with their pages, in no order."""
    seqs, page = case["seqs"], case["page"]
    count, length = _lengths(case)
    each = [-(-n // page) for n in length]
    total = sum(each)
    order = torch.randperm(total + 3, generator=gen, device="cuda")[:total].int()
    table = torch.full((seqs, max(each)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(each):
        table[b, :n] = order[at:at + n]
        at += n
    starts = torch.tensor([sum(count[:b]) for b in range(seqs + 1)], dtype=torch.int32)
    return dict(count=count, length=length, pool=total + 3, starts=starts.cuda(),
                lengths=torch.tensor(length, dtype=torch.int32).cuda(), pages=table)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt, hq, hk, dim = case["op"], case["dtype"], case["hq"], case["hk"], case["dim"]
    s = dict(case=case)
    paged = op in ("append", "attend")
    if paged:
        s["batch"] = batch = _batch(case, gen)
        tokens = sum(batch["count"])
        shape = (batch["pool"], case["page"], hk, dim)
        s["k_pages"], s["v_pages"] = (torch.randn(shape, generator=gen, device="cuda").to(TORCH[dt])
                                      for _ in range(2))
    else:
        tokens = case["tokens"]
        s["positions"] = torch.randint(case["far"], (tokens,), generator=gen, device="cuda") if "token" in \
            case.get("name", "") else torch.arange(tokens, device="cuda") % case["far"]
    if op == "attend":   # queries that prefer some keys to others
        s["q"] = (1.5 * torch.randn(tokens, hq, dim, generator=gen, device="cuda")).to(TORCH[dt])
    else:
        qkv = _projection(gen, tokens, hq + 2 * hk, dim, dt)
        s["q"], s["k"], s["v"] = qkv.split([hq, hk, hk], 1)
        if op.startswith("norm") or case.get("norm"):
            s["wq"], s["wk"] = (1 + 0.2 * torch.randn(dim, generator=gen, device="cuda") for _ in range(2))
        if op.endswith("step") or op.endswith("grad"):
            s["dq"], s["dk"] = ((0.1 * torch.randn(tokens, h, dim, generator=gen, device="cuda")).to(TORCH[dt])
                                for h in (hq, hk))
    if own:   # what a program makes once for its layer, and for a batch
        import pipelined_elementwise_streaming_gb300 as tsx

        if op != "attend":
            s["rotary"] = tsx.Rotary(dt, hq, hk, dim, rot=case["rot"], layout=case["layout"],
                                     scaling=_scaling(case), norm="rms" if "wq" in s else None, eps=EPS)
        if paged:
            s["attention"] = tsx.PagedAttention(dt, hq, hk, dim, case["page"], rotary=s.get("rotary"))
            s["cache"] = (s["k_pages"], s["v_pages"])
            s["tsx_batch"] = tsx.Batch(batch["starts"], batch["lengths"], batch["pages"], max(batch["count"]))
    return s


# ------------------------------------------------------------- plain form


def _frequencies(case):
    rot = case["rot"]
    i = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot
    base, amplitude, scaling = 10000.0, 1.0, _scaling(case)
    if scaling and scaling[0] == "ntk" and rot > 2:
        base *= scaling[1] ** (rot / (rot - 2))
    f = base ** -i
    if scaling and scaling[0] == "linear":
        f = f / scaling[1]
    if scaling and scaling[0] == "yarn":
        _, factor, length = scaling
        lo, hi = (rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64, device="cuda") - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
        amplitude = 1 + 0.1 * math.log(factor)
    return f, amplitude


def _turn(x, positions, case, back=False):
    """x fp32 [tokens, heads, dim] turned, or turned back (the gradient)."""
    rot = case["rot"]
    f, amplitude = _frequencies(case)
    angle = positions.double()[:, None] * f
    c, s = (amplitude * torch.cos(angle)).float()[:, None], (amplitude * torch.sin(angle)).float()[:, None]
    if back:
        s = -s
    if case["layout"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _normed(x, w):
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r * w


def _normed_backward(d, x, w):
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    hat = x * r
    g = d * w
    return r * (g - hat * (g * hat).mean(-1, keepdim=True)), (d * hat).sum((0, 1))


def _plain_attend(s):
    case, batch = s["case"], s["batch"]
    hk, dim = case["hk"], case["dim"]
    group = case["hq"] // hk
    out = torch.empty_like(s["q"])
    at = 0
    for b, (n, length) in enumerate(zip(batch["count"], batch["length"])):
        ids = batch["pages"][b, : -(-length // case["page"])].long()
        keys, values = (t[ids].flatten(0, 1)[:length].float().transpose(0, 1) for t in (s["k_pages"], s["v_pages"]))
        q = (s["q"][at:at + n].float() * dim ** -0.5).unflatten(1, (hk, group)).permute(1, 0, 2, 3)
        hidden = torch.arange(length, device="cuda") > torch.arange(length - n, length, device="cuda")[:, None]
        x = (q.reshape(hk, n * group, dim) @ keys.transpose(1, 2)).unflatten(1, (n, group))
        x = x.masked_fill_(hidden[:, None], float("-inf"))
        p = torch.exp(x - x.amax(-1, keepdim=True))
        y = (p.flatten(1, 2) @ values).unflatten(1, (n, group)) / p.sum(-1, keepdim=True)
        out[at:at + n] = y.transpose(0, 1).flatten(1, 2).to(out.dtype)
        at += n
    return out


def _slots(batch, page):
    """(position, row of the flattened pages) of every new token."""
    starts, lengths, pages = (batch[n].long() for n in ("starts", "lengths", "pages"))
    tokens = sum(batch["count"])
    seq = torch.repeat_interleave(torch.arange(len(lengths), device="cuda"), starts.diff(), output_size=tokens)
    p = lengths[seq] - starts[seq + 1] + torch.arange(tokens, device="cuda")
    return p, pages[seq, p // page] * page + p % page


def _plain(s):
    case = s["case"]
    op, t = case["op"], TORCH[case["dtype"]]
    if op == "attend":
        return _plain_attend(s)
    q, k = s["q"].float(), s["k"].float()
    if op == "append":
        positions, rows = _slots(s["batch"], case["page"])
        if "wq" in s:
            q, k = _normed(q, s["wq"]), _normed(k, s["wk"])
        for pages, new in ((s["k_pages"], _turn(k, positions, case).to(t)), (s["v_pages"], s["v"])):
            pages.view(-1, *pages.shape[2:])[rows] = new
        return _turn(q, positions, case).to(t), s["k_pages"], s["v_pages"]
    positions, out = s["positions"], ()
    if not op.endswith("grad"):
        a, b = (q, k) if op.startswith("rotary") else (_normed(q, s["wq"]), _normed(k, s["wk"]))
        out = (_turn(a, positions, case).to(t), _turn(b, positions, case).to(t))
    if op in ("rotary", "norm"):
        return out
    dq, dk = (_turn(s[n].float(), positions, case, back=True) for n in ("dq", "dk"))
    if op == "rotary_step":
        return (*out, dq.to(t), dk.to(t))
    (dq, dwq), (dk, dwk) = _normed_backward(dq, q, s["wq"]), _normed_backward(dk, k, s["wk"])
    return (*out, dq.to(t), dk.to(t), dwq, dwk)


# -------------------------------------------------------------- the library


def _library(s):
    op = s["case"]["op"]
    if op == "attend":
        return s["attention"].forward(s["q"], s["cache"], s["tsx_batch"])
    if op == "append":
        q = s["attention"].append(s["q"], s["k"], s["v"], s["cache"], s["tsx_batch"], s.get("wq"), s.get("wk"))
        return (q, *s["cache"])
    f, weights, out = s["rotary"], (s.get("wq"), s.get("wk")), ()
    if not op.endswith("grad"):
        out = f.forward(s["q"], s["k"], s["positions"], *weights)
    if op in ("rotary", "norm"):
        return out
    if op == "rotary_step":
        return (*out, *f.backward(s["dq"], s["dk"], s["positions"]))
    return (*out, *f.backward(s["dq"], s["dk"], s["positions"], s["q"], s["k"], *weights))


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------ what it needs


def work(case):
    """Each input read once, each output written once; of a cache what the
    call has to read or write."""
    op, es, hq, hk, dim = case["op"], SIZE[case["dtype"]], case["hq"], case["hk"], case["dim"]
    if op == "attend":
        count, length = _lengths(case)
        pairs = sum(n * (m - (n - 1) / 2) for n, m in zip(count, length))
        return {"bytes": es * dim * 2 * (hk * sum(length) + hq * sum(count)), "flops": 4 * dim * hq * int(pairs)}
    if op == "append":
        tokens = sum(_lengths(case)[0])
        return {"bytes": 2 * es * tokens * dim * (hq + 2 * hk), "flops": 8 * tokens * (hq + hk) * dim}
    e = case["tokens"] * (hq + hk) * dim
    passes = {"rotary": 2, "norm": 2, "rotary_step": 4, "norm_step": 5, "norm_grad": 3}[op]
    flops = {"rotary": 3, "norm": 6, "rotary_step": 6, "norm_step": 20, "norm_grad": 14}[op]
    return {"bytes": passes * es * e + 8 * case["tokens"], "flops": flops * e}


# --------------------------------------------------------- 64-bit definition


def _phases64(case, positions):
    """amplitude * exp(i angle), complex [tokens, rot / 2]"""
    rot, how = case["rot"], case["scaling"]
    f, size = [], 1.0
    for j in range(rot // 2):
        e = 2 * j / rot
        w = 10000.0 ** -e
        if how == "linear":
            w /= 4
        elif how == "ntk" and rot > 2:
            w *= 4.0 ** (-2 * j / (rot - 2))
        elif how == "yarn":
            def bound(turns):
                return rot / 2 * math.log(32768 / (2 * math.pi * turns), 10000.0)

            first, last = max(math.floor(bound(32)), 0), min(math.ceil(bound(1)), rot - 1)
            slow = min(max((j - first) / max(last - first, 1e-3), 0.0), 1.0)
            w *= (1 - slow) + slow / 16
            size = 0.1 * math.log(16) + 1
        f.append(w)
    angle = torch.outer(positions.double(), torch.tensor(f, dtype=torch.float64, device="cuda"))
    return torch.polar(torch.full_like(angle, size), angle)


def _turn64(x, z, layout):
    """x fp64 [tokens, heads, dim] with its pairs as complex numbers times z."""
    rot = 2 * z.shape[1]
    out = x.clone()
    head = x[..., :rot].unflatten(-1, (2, rot // 2)) if layout == "half" else \
        x[..., :rot].unflatten(-1, (rot // 2, 2)).transpose(-1, -2)
    w = torch.complex(head[..., 0, :].contiguous(), head[..., 1, :].contiguous()) * z[:, None]
    if layout == "half":
        out[..., : rot // 2], out[..., rot // 2: rot] = w.real, w.imag
    else:
        out[..., 0:rot:2], out[..., 1:rot:2] = w.real, w.imag
    return out


def _hat64(x):
    """(x rstd, rstd)"""
    r = (torch.einsum("thd,thd->th", x, x) / x.shape[-1] + EPS) ** -0.5
    return x * r[..., None], r


def _attend64(s):
    case, batch = s["case"], s["batch"]
    hk, dim, page = case["hk"], case["dim"], case["page"]
    out, at = [], 0
    for b, (n, length) in enumerate(zip(batch["count"], batch["length"])):
        table = batch["pages"][b].tolist()
        k, v = (torch.cat([t[table[i]] for i in range(-(-length // page))])[:length].double()
                for t in (s["k_pages"], s["v_pages"]))
        q = s["q"][at:at + n].double().unflatten(1, (hk, -1))
        mine = torch.empty_like(q)
        for first in range(0, n, 128):
            part = q[first:first + 128]
            last = length - n + first + torch.arange(part.shape[0], device="cuda")
            for h in range(hk):
                x = torch.einsum("tgd,kd->tgk", part[:, h], k[:, h]) / math.sqrt(dim)
                x[(torch.arange(length, device="cuda") > last[:, None])[:, None].expand_as(x)] = -math.inf
                weight = torch.exp(x - torch.logsumexp(x, -1, keepdim=True))
                mine[first:first + 128, h] = torch.einsum("tgk,kd->tgd", weight, v[:, h])
        out.append(mine.flatten(1, 2))
        at += n
    return torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    op, layout = case["op"], case.get("layout")
    if op == "attend":
        return _attend64(s)
    q, k = s["q"].double(), s["k"].double()
    a, b = q, k
    if "wq" in s:
        (hq, rq), (hk, rk) = _hat64(q), _hat64(k)
        a, b = hq * s["wq"].double(), hk * s["wk"].double()
    if op == "append":
        batch, page = s["batch"], case["page"]
        caches = [s["k_pages"].double(), s["v_pages"].double()]
        places = [(b, length - n + j) for b, (n, length) in enumerate(zip(batch["count"], batch["length"]))
                  for j in range(n)]
        table = batch["pages"].tolist()
        z = _phases64(case, torch.tensor([p for _, p in places], device="cuda"))
        ids = torch.tensor([table[i][p // page] for i, p in places], device="cuda")
        slots = torch.tensor([p % page for _, p in places], device="cuda")
        caches[0].index_put_((ids, slots), _turn64(b, z, layout))
        caches[1].index_put_((ids, slots), s["v"].double())
        return (_turn64(a, z, layout), *caches)
    z = _phases64(case, s["positions"])
    out = (_turn64(a, z, layout), _turn64(b, z, layout))
    if op in ("rotary", "norm"):
        return out
    grads = [_turn64(s[name].double(), z.conj(), layout) for name in ("dq", "dk")]
    if op == "rotary_step":
        return (*out, *grads)
    dx, dw = [], []
    for g, hat, r, w in ((grads[0], hq, rq, s["wq"]), (grads[1], hk, rk, s["wk"])):
        gw = g * w.double()
        along = torch.einsum("thd,thd->th", gw, hat) / gw.shape[-1]
        dx.append((gw - along[..., None] * hat) * r[..., None])
        dw.append(torch.einsum("thd,thd->d", g, hat))
    return (*(out if op == "norm_step" else ()), *dx, *dw)
