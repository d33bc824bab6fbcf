"""The layer operators (include/tsx_layers.h) against their definitions in 64
bits (oracle/layers.py).

Tolerances.  u = 2^-24 is fp32's rounding, ut the element type's (2^-11, 2^-8,
2^-24); sums of k terms carry at most gamma(k) = k u / (1 - k u) of the sum of
magnitudes whatever the order; the sigmoid's relative error is under SIG =
2^-18 (16-bit data: ex2.approx and rcp.approx, a few ulps each) or 2^-20 (fp32:
expf and a division; the argument's rounding adds |z| u).  The bounds below put
these through the formulas, element by element.
"""

import numpy as np
import pytest

from oracle import layers as ref
from tests import _gpu
from tests._gpu import torch

pytestmark = pytest.mark.gpu

U = 2.0**-24
UT = {"f16": 2.0**-11, "bf16": 2.0**-8, "f32": 2.0**-24}
TINY = {"f16": 2.0**-24, "bf16": 2.0**-126, "f32": 2.0**-126}   # spacing of the smallest numbers, or below
SIG = {"f16": 2.0**-18, "bf16": 2.0**-18, "f32": 2.0**-20}
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DTYPES = ["f16", "bf16", "f32"]


@pytest.fixture(scope="module")
def tsx():
    _gpu.need_gpu()
    import pipelined_elementwise_streaming_gb300 as m

    return m


def gamma(k):
    return k * U / (1 - k * U)


def dev(a, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda").to(TORCH[dtype])


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def values(shape, dtype, seed, scale=1.0, offset=0.0):
    """(CUDA tensor of the type, its exact values in 64 bits)"""
    rng = np.random.default_rng(seed)
    t = dev(rng.standard_normal(shape) * scale + offset, dtype)
    return t, host(t)


def sliced(t, pitch):
    """The same values in rows `pitch` elements apart, NaN between them."""
    wide = torch.full((*t.shape[:-1], pitch), float("nan"), dtype=t.dtype, device=t.device)
    wide[..., : t.shape[-1]] = t
    return wide[..., : t.shape[-1]]


def within(got, want, bound, what):
    got = host(got) if torch.is_tensor(got) else got
    assert got.shape == want.shape, what
    off = np.abs(got - want) - bound
    k = np.unravel_index(np.argmax(off), off.shape) if off.size else None
    assert not off.size or off[k] <= 0, f"{what}: at {k}: got {got[k]!r} want {want[k]!r} bound {bound[k]!r}"
    assert np.array_equal(np.isnan(got), np.isnan(want)), what


def rounded(want, e, dtype):
    """Bound of a value computed within e and rounded into the type."""
    return 1.001 * (e + UT[dtype] * (np.abs(want) + e)) + TINY[dtype]


def act_error(z, ez, kind, dtype):
    """Errors of act(z) and act'(z) for z within ez: |act'| < 1.2, |act''| <
    1.2, and the sigmoid's own error, which z and z' s argument amplify."""
    if kind == "none":
        return ez, np.zeros_like(ez)
    s = SIG[dtype] + 8 * U * (1 + np.abs(z))
    return 1.2 * ez + np.abs(z) * s, 1.2 * ez + 4 * (1 + np.abs(z)) * s


def norm_errors(x, w, b, mean, rstd, groups, eps):
    """Errors of mean, rstd, xhat and z as the kernels form them."""
    n, l, c = x.shape
    per = c // groups
    m = l * per
    v = np.abs(x).reshape(n, l, groups, per)
    e_mean = gamma(m + 8) * v.mean((1, 3)) + 1e-40
    # squared deviations are positive: a relative gamma, plus the square of the mean's own error
    e_rstd = rstd * (gamma(m + 16) + 0.5 * (e_mean * rstd) ** 2 + 4 * U)
    em, er, mu, rs = (np.repeat(t, per, 1)[:, None, :] for t in (e_mean, e_rstd, mean, rstd))
    hat = (x - mu) * rs
    e_hat = rs * (em + 2 * U * (np.abs(x) + np.abs(mu))) + np.abs(hat) * (er / rs + 2 * U)
    z = hat * w + b
    return e_mean, e_rstd, hat, e_hat, z, np.abs(w) * e_hat + 3 * U * (np.abs(hat * w) + np.abs(b))


# n, l, c, groups: one token; heads of tokens; groups of 1, 4, 10 channels; odd everything; one group; a group
# wider than a CTA's row; rows cut into several runs; one channel; long samples cut into ranges
NORM_SHAPES = [
    (1, 1, 64, 4), (37, 1, 4096, 32), (5, 1, 96, 12), (3, 7, 24, 24), (2, 33, 128, 32), (2, 100, 320, 32),
    (3, 29, 198, 11), (2, 5, 30, 1), (4, 1, 2560, 1), (2, 3, 6000, 2), (1, 40, 5120, 40), (9, 13, 1, 1),
    (1, 3001, 64, 8), (1, 1500, 33, 3), (300, 2, 40, 5), (2, 1, 8208, 2), (1, 2, 4097, 1),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_norm_and_its_gradient(tsx, shape, dtype):
    n, l, c, groups = shape
    for k, act in enumerate(("none", "silu", "gelu")):
        check_norm(tsx, n, l, c, groups, dtype, act, seed=1000 * k + n + l + c)


# what decides how a call runs: tokens whose groups lie within a warp (and not); small samples side by side in a CTA;
# samples shared by clusters of 2, 8 and 16 CTAs, with ranks left without rows; samples only just too long for that
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [
    (3000, 1, 512, 8), (40, 1, 1280, 5), (3, 1, 4096, 2), (9, 1, 24, 3), (700, 3, 64, 8), (900, 7, 320, 32),
    (2000, 2, 16, 16), (1, 1000, 2048, 1), (1, 100, 2048, 1), (2, 4000, 64, 4), (1, 8192, 64, 2), (1, 8200, 64, 64),
    (1, 17, 2048, 2048), (16, 300, 96, 4), (3, 512, 640, 32),
    (1, 5000, 2048, 2048), (1, 9000, 320, 320), (2, 3000, 1000, 1), (1, 20000, 24, 3), (600, 200, 64, 4),
], ids=lambda s: "x".join(map(str, s)))
def test_norm_however_it_runs(tsx, shape, dtype):
    n, l, c, groups = shape
    check_norm(tsx, n, l, c, groups, dtype, "silu", seed=n + l + c)


def check_norm(tsx, n, l, c, groups, dtype, act, seed, offset=0.3, x_pitch=None, y_pitch=None, param="f32", eps=1e-5,
               form="int8", block=128):
    x, x64 = values((n, l, c), dtype, seed, 1.5, offset)
    w, w64 = values((c,), param, seed + 1, 0.3, 1.0)
    b, b64 = values((c,), param, seed + 2, 0.3)
    dy, dy64 = values((n, l, c), dtype, seed + 3)
    if x_pitch:
        x = sliced(x, x_pitch)
    if y_pitch:
        dy = sliced(dy, y_pitch)
    op = tsx.GroupNorm(dtype, n, l, c, groups, act=act, eps=eps, x_pitch=x_pitch, y_pitch=y_pitch, param_dtype=param,
                       form=form, block=block)
    y, mean, rstd = op.forward(x, w, b)
    want, mean64, rstd64 = ref.norm(x64, w64, b64, groups, act, eps)
    em, er, hat, e_hat, z, ez = norm_errors(x64, w64, b64, mean64, rstd64, groups, eps)
    what = f"{dtype} {act} {(n, l, c, groups)}"
    within(mean, mean64, em, what + " mean")
    within(rstd, rstd64, er, what + " rstd")
    ev, _ = act_error(z, ez, act, dtype)
    within(y, want, rounded(want, ev, dtype), what + " y")

    y2, mean2, rstd2, saved = op.forward(x, w, b, checkpoint=True)
    for p, q in ((y, y2), (mean, mean2), (rstd, rstd2)):
        # another layout of runs may add in another order: the same bounds hold
        within(q, want if p is y else mean64 if p is mean else rstd64,
               rounded(want, ev, dtype) if p is y else em if p is mean else er, what + " with the checkpoint")
    check_held(saved, host(x).reshape(n * l, c), form, block, what)

    # the gradient at the statistics given, so their error is none of its own
    m64, r64 = host(mean), host(rstd)
    for src, xs in ((x, x64), (saved, ref.stands_for(held_numbers(saved), saved.scale.cpu().numpy(), block).reshape(
            n, l, c))):
        dx, dw, db = op.backward(dy, src, w, b, mean, rstd)
        check_norm_gradient(dx, dw, db, dy64, xs, w64, b64, m64, r64, groups, act, dtype, what)


def check_norm_gradient(dx, dw, db, dy, x, w, b, mean, rstd, groups, act, dtype, what):
    n, l, c = x.shape
    per = c // groups
    mu, rs = (np.repeat(t, per, 1)[:, None, :] for t in (mean, rstd))
    hat = (x - mu) * rs
    # x itself carries one rounding from a checkpoint
    e_hat = 4 * U * np.abs(hat) + 2 * U * np.abs(x) * rs
    z = hat * w + b
    ez = np.abs(w) * e_hat + 3 * U * (np.abs(hat * w) + np.abs(b))
    slope = ref.act(z, act)[1]
    dz = dy * slope
    e_dz = np.abs(dy) * (act_error(z, ez, act, dtype)[1] + 2 * U * np.abs(slope))
    wdx, wdw, wdb = ref.norm_backward(dy, x, w, b, mean, rstd, groups, act)

    def over_group(v):
        return np.repeat(v.reshape(n, l, groups, per).mean((1, 3)), per, 1)[:, None, :]

    e_prod = e_dz * np.abs(hat) + np.abs(dz) * (e_hat + U * np.abs(hat))
    g = gamma(l * per + 16)
    aw = np.abs(w)
    s1 = over_group(aw * (e_dz + g * np.abs(dz)))
    s2 = over_group(aw * (e_prod + g * np.abs(dz * hat)))
    m2 = np.abs(over_group(dz * w * hat))
    e = rs * (aw * e_dz + s1 + np.abs(hat) * s2 + e_hat * m2 +
              4 * U * (np.abs(dz * w) + np.abs(over_group(dz * w)) + np.abs(hat) * m2))
    within(dx, wdx, rounded(wdx, e, dtype), what + " dx")
    g = gamma(n * l + 16)
    within(dw, wdw, (e_prod + g * np.abs(dz * hat)).sum((0, 1)) * 1.001 + 1e-37, what + " dweight")
    within(db, wdb, (e_dz + g * np.abs(dz)).sum((0, 1)) * 1.001 + 1e-37, what + " dbias")


def held_numbers(saved):
    return host(saved.q)


def check_held(saved, x, form, block, what):
    q, scale = ref.hold(x, form, block)
    got = saved.scale.cpu().numpy()
    assert np.array_equal(got, scale, equal_nan=True), what + " scales"
    bad = np.nonzero(held_numbers(saved) != q)
    assert bad[0].size == 0, f"{what}: number at {[int(i[0]) for i in bad]} differs"


@pytest.mark.parametrize("dtype,param", [("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("form,block", [("int8", 32), ("int8", 64), ("e4m3", 128), ("e4m3", 32)])
def test_norm_parameters_pitches_and_forms(tsx, dtype, param, form, block):
    check_norm(tsx, 2, 19, 192, 6, dtype, "silu", 5, x_pitch=200, y_pitch=256, param=param, form=form, block=block)
    check_norm(tsx, 3, 11, 130, 13, dtype, "gelu", 6, x_pitch=131, y_pitch=130, param=param, form=form, block=block)


@pytest.mark.parametrize("shape", [(3001, 1, 512, 8), (40, 30, 64, 8), (2, 3000, 64, 4), (1, 1000, 320, 32)],
                         ids=lambda s: "x".join(map(str, s)))
def test_norm_of_rows_that_start_half_a_sector_apart(tsx, shape):
    """fp32 rows that are aligned to 16 bytes, every other one to 32."""
    n, l, c, groups = shape
    check_norm(tsx, n, l, c, groups, "f32", "silu", 7, x_pitch=c + 4, y_pitch=c + 12)


def test_norm_of_a_large_mean_keeps_its_digits(tsx):
    """Mean 1000, spread 1: E[x^2] - mean^2 in fp32 would leave an error of
    about 1000^2 2^-24 = 6 % in the variance.  Here it has to be as exact as
    the mean, whose error of gamma A costs its square only."""
    for shape in ((2, 64, 96, 4), (64, 1, 1024, 8), (1, 5000, 32, 2)):
        n, l, c, groups = shape
        x, x64 = values((n, l, c), "f32", 3, 1.0, 1000.0)
        one, zero = dev(np.ones(c)), dev(np.zeros(c))
        _, mean, rstd = tsx.GroupNorm("f32", n, l, c, groups).forward(x, one, zero)
        _, m64, r64 = ref.norm(x64, np.ones(c), np.zeros(c), groups, "none", 1e-5)
        assert np.abs(host(rstd) / r64 - 1).max() < 2e-5
        assert np.abs(host(mean) / m64 - 1).max() < 1e-6


def test_norm_of_constant_groups(tsx):
    n, l, c, groups = 2, 9, 48, 3
    x = dev(np.full((n, l, c), 7.0), "bf16")
    w, b = dev(np.ones(c)), dev(np.full(c, 0.5))
    y, mean, rstd = tsx.GroupNorm("bf16", n, l, c, groups).forward(x, w, b)
    assert torch.all(mean == 7) and torch.all(y == 0.5)
    assert np.abs(host(rstd) * np.sqrt(1e-5) - 1).max() < 1e-6


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("shape", [(3, 1, 256, 8), (2, 50, 96, 6), (2, 7, 33, 3)])
def test_norm_not_finite_stays_in_its_group(tsx, bad, shape):
    n, l, c, groups = shape
    x, _ = values((n, l, c), "bf16", 8)
    x[1, l // 2, 5] = bad
    w, b = dev(np.ones(c)), dev(np.zeros(c))
    op = tsx.GroupNorm("bf16", n, l, c, groups, act="silu")
    clean = x.clone()
    clean[1, l // 2, 5] = 0
    y, mean, rstd, saved = op.forward(x, w, b, checkpoint=True)
    y0, _, _ = op.forward(clean, w, b)
    inside = torch.zeros_like(x, dtype=torch.bool)
    inside[1, :, : c // groups] = True
    assert torch.isnan(y[inside]).all()
    assert torch.equal(y[~inside], y0[~inside])
    # the checkpoint's block reads back as NaN, and so does the group's gradient
    assert torch.isnan(saved.scale[l + l // 2, 0]) and torch.isnan(saved.scale).sum() == 1
    dx, _, _ = op.backward(clean, saved, w, b, mean, rstd)
    assert torch.isnan(dx[1, l // 2, 5])


def test_norm_in_place_and_repeated_bit_for_bit(tsx):
    for n, l, c, groups in ((16, 1, 512, 8), (2, 200, 320, 32), (2, 7000, 64, 4), (3, 50, 33, 3)):
        x, _ = values((n, l, c), "bf16", 9)
        w, b = values((c,), "f32", 10, 0.2, 1)[0], values((c,), "f32", 11)[0]
        dy, _ = values((n, l, c), "bf16", 12)
        op = tsx.GroupNorm("bf16", n, l, c, groups, act="silu")
        y, mean, rstd = op.forward(x, w, b)
        dx, dw, db = op.backward(dy, x, w, b, mean, rstd)
        for _ in range(3):
            again = op.forward(x, w, b)
            assert all(torch.equal(p, q) for p, q in zip(again, (y, mean, rstd)))
            again = op.backward(dy, x, w, b, mean, rstd)
            assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))
        z = x.clone()
        op.forward(z, w, b, out=z)
        assert torch.equal(z, y)
        g = dy.clone()
        op.backward(g, x, w, b, mean, rstd, out=g)
        assert torch.equal(g, dx)


def test_norm_gradient_against_differences(tsx):
    """Directional derivatives of sum(dy y) by central differences of the
    64-bit forward pass, step 1e-5 (error of order 1e-10 relative to third
    derivatives of order 1), against the fp32 gradients, whose sums of at most
    2e3 terms carry under gamma(2e3) = 1.2e-4 of their magnitudes."""
    for act in ("none", "silu", "gelu"):
        n, l, c, groups, eps = 2, 9, 40, 5, 1e-3
        (x, x64), (dy, dy64) = values((n, l, c), "f32", 20), values((n, l, c), "f32", 21)
        (w, w64), (b, b64) = values((c,), "f32", 22, 0.3, 1), values((c,), "f32", 23, 0.3)
        op = tsx.GroupNorm("f32", n, l, c, groups, act=act, eps=eps)
        _, mean, rstd = op.forward(x, w, b)
        grads = [host(t) for t in op.backward(dy, x, w, b, mean, rstd)]
        rng = np.random.default_rng(24)
        for k, at in enumerate((x64, w64, b64)):
            v = rng.standard_normal(at.shape)
            args = [x64, w64, b64]

            def loss(t):
                args[k] = at + t * v
                return (dy64 * ref.norm(*args, groups, act, eps)[0]).sum()

            slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
            assert abs((grads[k] * v).sum() - slope) <= 1.2e-4 * np.abs(grads[k] * v).sum() + 1e-6, (act, k)


def test_norm_without_rows(tsx):
    w, b = dev(np.ones(16)), dev(np.zeros(16))
    op = tsx.GroupNorm("bf16", 3, 0, 16, 4)
    x = torch.empty(3, 0, 16, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = op.forward(x, w, b)
    assert y.shape == x.shape and torch.all(mean == 0) and np.allclose(host(rstd), 1e-5**-0.5)
    for n, l in ((3, 0), (0, 5)):
        op = tsx.GroupNorm("bf16", n, l, 16, 4)
        x = torch.empty(n, l, 16, dtype=torch.bfloat16, device="cuda")
        stats = torch.zeros(n, 4, device="cuda")
        assert op.forward(x, w, b)[0].shape == x.shape
        dx, dw, db = op.backward(x, x, w, b, stats, stats)
        assert dx.shape == x.shape and torch.all(dw == 0) and torch.all(db == 0)


# --------------------------------------------------------- gated activation

GATED_SHAPES = [(1, 1), (1, 8), (3, 17), (7, 128), (33, 200), (5, 1000), (64, 4096), (2, 11009), (130, 72)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", GATED_SHAPES)
def test_gated_and_its_gradient(tsx, rows, cols, dtype):
    for k, (act, form, block) in enumerate((("silu", "int8", 128), ("gelu", "e4m3", 64), ("none", "int8", 32))):
        check_gated(tsx, rows, cols, dtype, act, form, block, 10 * k + rows + cols)
    check_gated(tsx, rows, cols, dtype, "silu", "int8", 128, 3, in_pitch=2 * cols + 5, out_pitch=cols + 3)
    check_gated(tsx, rows, cols, dtype, "silu", "e4m3", 32, 4, in_pitch=2 * cols + 8, out_pitch=cols + 8)


def check_gated(tsx, rows, cols, dtype, act, form, block, seed, in_pitch=None, out_pitch=None):
    (g, g64), (u, u64) = values((rows, cols), dtype, seed, 2), values((rows, cols), dtype, seed + 1)
    dh, dh64 = values((rows, cols), dtype, seed + 2)
    if in_pitch:
        both = torch.full((rows, in_pitch), float("nan"), dtype=g.dtype, device="cuda")
        both[:, :cols], both[:, cols: 2 * cols] = g, u
        g, u = both[:, :cols], both[:, cols: 2 * cols]
    if out_pitch:
        dh = sliced(dh, out_pitch)
    op = tsx.GatedAct(dtype, rows, cols, act=act, form=form, block=block, in_pitch=in_pitch, out_pitch=out_pitch)
    what = f"{dtype} {act} {(rows, cols, in_pitch)}"

    def check_h(h, a, b, ea, eb):
        value, _ = ref.act(a, act)
        ev = act_error(a, ea, act, dtype)[0]
        want = value * b
        within(h, want, rounded(want, ev * np.abs(b) + np.abs(value) * eb + 2 * U * np.abs(want), dtype), what + " h")

    none = np.zeros_like(g64)
    check_h(op.forward(g, u), g64, u64, none, none)
    h, cg, cu = op.forward(g, u, checkpoint=True)
    check_h(h, g64, u64, none, none)
    check_held(cg, g64, form, block, what + " gate")
    check_held(cu, u64, form, block, what + " up")
    a64, b64 = (ref.stands_for(held_numbers(c), c.scale.cpu().numpy(), block) for c in (cg, cu))
    for (sg, su), a, b, e in (((g, u), g64, u64, 0), ((cg, cu), a64, b64, U)):
        dg, du, h = op.backward(dh, sg, su, recompute=True)
        plain = op.backward(dh, sg, su)
        assert torch.equal(plain[0], dg) and torch.equal(plain[1], du)
        ea, eb = e * np.abs(a), e * np.abs(b)
        check_h(h, a, b, ea, eb)
        value, slope = ref.act(a, act)
        ev, es = act_error(a, ea, act, dtype)
        wg, wu = ref.gated_backward(dh64, a, b, act)
        within(dg, wg, rounded(wg, np.abs(dh64) * (np.abs(b) * es + eb * np.abs(slope)) + 3 * U * np.abs(wg), dtype),
               what + " dgate")
        within(du, wu, rounded(wu, np.abs(dh64) * ev + 2 * U * np.abs(wu), dtype), what + " dup")


def test_gated_gradient_against_differences(tsx):
    rows, cols = 5, 24
    (g, g64), (u, u64), (dh, dh64) = (values((rows, cols), "f32", 30 + k) for k in range(3))
    for act in ("silu", "gelu"):
        dg, du = tsx.GatedAct("f32", rows, cols, act=act).backward(dh, g, u)
        rng = np.random.default_rng(33)
        for k, grad in enumerate((host(dg), host(du))):
            v = rng.standard_normal((rows, cols))

            def loss(t):
                return (dh64 * ref.gated(g64 + t * v * (k == 0), u64 + t * v * (k == 1), act)).sum()

            slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
            assert abs((grad * v).sum() - slope) <= 1e-5 * np.abs(grad * v).sum() + 1e-8


def test_gated_extremes(tsx):
    """Very large and infinite arguments: values are their limits, no NaN
    where the formula has none."""
    z = np.array([[-3e38, -1e30, -1e4, -100, -30, -0.0, 0.0, 30, 100, 1e4, 1e30, 3e38]])
    g, one = dev(z), dev(np.ones_like(z))
    z = host(g)   # as fp32 holds them
    for act in ("silu", "gelu"):
        op = tsx.GatedAct("f32", 1, z.size, act=act)
        h = host(op.forward(g, one))
        dg, du = (host(t) for t in op.backward(one, g, one))
        big = np.abs(z) > 99
        assert np.array_equal(h[big], np.where(z > 0, z, 0.0)[big])
        assert np.array_equal(dg[big], (z > 0).astype(float)[big])
        assert np.array_equal(du, h)
        assert np.all(np.isfinite(dg)) and np.all(np.isfinite(h))
    nan = tsx.GatedAct("f32", 1, 1, act="gelu").forward(dev([[np.nan]]), dev([[1.0]]))
    assert torch.isnan(nan).all()


# ------------------------------------------------------------- checkpoints


def test_gated_rows_that_start_half_a_sector_apart(tsx):
    check_gated(tsx, 33, 200, "f32", "gelu", "int8", 64, 8, in_pitch=412, out_pitch=204)
    check_gated(tsx, 7, 4096, "f32", "silu", "e4m3", 32, 9, in_pitch=8196, out_pitch=4100)


def test_pack_of_rows_that_start_half_a_sector_apart(tsx):
    x = dev(values((19, 1032), "f32", 3)[1], "f32")
    wide = sliced(x, 1036)
    for form in ("int8", "e4m3"):
        op = tsx.Packer("f32", 19, 1032, form=form, block=128, pitch=1036)
        saved = op.pack(wide)
        check_held(saved, host(x), form, 128, form)
        dense = tsx.Packer("f32", 19, 1032, form=form, block=128).unpack(saved)
        assert torch.equal(op.unpack(saved), dense)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("block", [32, 64, 128])
def test_pack_and_unpack(tsx, dtype, form, block):
    for rows, cols, pitch in ((1, 1, None), (3, 7, None), (2, 33, 40), (5, 128, None), (9, 200, 208), (4, 129, None),
                              (17, 4096, None), (3, 5000, 5001), (2, 12345, None)):
        x, x64 = values((rows, cols), dtype, rows + cols, 3.0)
        x64 = x64 * np.exp2(np.random.default_rng(cols).integers(-12, 5, cols))   # columns of many magnitudes
        x = dev(x64, dtype)
        x64 = host(x)
        src = sliced(x, pitch) if pitch else x
        op = tsx.Packer(dtype, rows, cols, form=form, block=block, pitch=pitch)
        saved = op.pack(src)
        what = f"{dtype} {form} {block} {(rows, cols, pitch)}"
        check_held(saved, x64, form, block, what)
        back = op.unpack(saved)
        want = ref.stands_for(held_numbers(saved), saved.scale.cpu().numpy(), block)
        within(back, want, rounded(want, U * np.abs(want), dtype), what + " back")
        # the error that the header states
        scale = np.repeat(saved.scale.cpu().numpy().astype(np.float64), block, 1)[:, :cols]
        step = 0.5 * scale if form == "int8" else np.maximum(2.0**-4 * np.abs(x64), scale / 1024)
        assert np.all(np.abs(want - x64) <= step * (1 + 1e-5) + 1e-6 * np.abs(x64))


def test_pack_of_special_blocks(tsx):
    for form in ("int8", "e4m3"):
        x = np.ones((6, 96), np.float32)
        x[0, :32] = 0                         # zeros
        x[1, :32] = 2.0**-121                 # below what a block keeps
        x[2, 40] = np.inf
        x[3, 41] = np.nan
        x[4, 70] = -3e38                      # the type's far end
        x[5, :32] = 2.0**-119                 # the smallest kept
        for dtype in ("f32", "bf16"):
            t = dev(x, dtype)
            op = tsx.Packer(dtype, 6, 96, form=form, block=32)
            saved = op.pack(t)
            check_held(saved, host(t), form, 32, f"{form} {dtype}")
            back = host(op.unpack(saved))
            assert np.all(back[0, :32] == 0) and np.all(back[1, :32] == 0)
            assert np.isnan(back[2, 32:64]).all() and np.isnan(back[3, 32:64]).all()
            assert np.isfinite(back[[0, 1, 4, 5]]).all() and np.isfinite(back[2, 64:]).all()


def test_pack_repeats_itself_exactly(tsx):
    """What a checkpoint reads back as packs to the same numbers again: the
    largest magnitude is among them."""
    x, _ = values((16, 512), "f32", 40)
    op = tsx.Packer("f32", 16, 512)
    first = op.pack(x)
    second = op.pack(op.unpack(first))
    assert torch.equal(first.q, second.q)


def test_offsets_past_32_bits(tsx):
    """More than 2^31 elements: the last rows are as the first of a small
    tensor."""
    rows, cols = (1 << 31) // 16384 + 5, 16384
    small, _ = values((5, cols), "bf16", 41)
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-5:] = small
    saved = tsx.Packer("bf16", rows, cols).pack(x)
    want = tsx.Packer("bf16", 5, cols).pack(small)
    assert torch.equal(saved.q[-5:], want.q) and torch.equal(saved.scale[-5:], want.scale)
    assert torch.equal(saved.q[:5], torch.zeros_like(want.q))
    x.fill_(1.0)
    tsx.Packer("bf16", rows, cols).unpack(saved, out=x)
    assert torch.equal(x[-5:], tsx.Packer("bf16", 5, cols).unpack(want))
    del saved
    # group norm with one sample past the boundary
    w, b = dev(np.ones(cols)), dev(np.zeros(cols))
    x[-5:] = small
    y, mean, rstd = tsx.GroupNorm("bf16", rows, 1, cols, 128).forward(x.view(rows, 1, cols), w, b)
    y5, mean5, rstd5 = tsx.GroupNorm("bf16", 5, 1, cols, 128).forward(small.view(5, 1, cols), w, b)
    assert torch.equal(y[-5:], y5) and torch.equal(mean[-5:], mean5) and torch.equal(rstd[-5:], rstd5)


# -------------------------------------------------------- calls and errors


def test_outputs_stay_inside_their_rows(tsx):
    """NaN canaries between and around rows are not written."""
    rows, cols, pitch = 6, 40, 56
    for off in (0, 1, 8):
        flat = torch.full((rows * pitch + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
        view = flat[off: off + rows * pitch].view(rows, pitch)[:, :cols]
        x, _ = values((rows, cols), "bf16", 50)
        tsx.GatedAct("bf16", rows, cols, out_pitch=pitch).forward(x, x, out=view)
        assert torch.isnan(flat).sum() == flat.numel() - rows * cols
        flat.fill_(float("nan"))
        w, b = dev(np.ones(cols)), dev(np.zeros(cols))
        tsx.GroupNorm("bf16", 2, 3, cols, 5, y_pitch=pitch).forward(x.view(2, 3, cols), w, b,
                                                                    out=view.unflatten(0, (2, 3)))
        assert torch.isnan(flat).sum() == flat.numel() - rows * cols


def test_other_streams_and_graphs(tsx):
    n, l, c, groups = 4, 300, 256, 8
    x, _ = values((n, l, c), "bf16", 60)
    dy, _ = values((n, l, c), "bf16", 61)
    w, b = dev(np.ones(c)), dev(np.zeros(c))
    norm = tsx.GroupNorm("bf16", n, l, c, groups, act="silu")
    glu = tsx.GatedAct("bf16", n * l, c)
    flat = x.view(n * l, c)

    def step(stream=None):
        y, mean, rstd, saved = norm.forward(x, w, b, checkpoint=True, stream=stream)
        h, cg, cu = glu.forward(flat, y.view(n * l, c), checkpoint=True, stream=stream)
        dg, du = glu.backward(h, cg, cu, stream=stream)
        return (y, mean, rstd, h, dg, du, *norm.backward(dy, saved, w, b, mean, rstd, stream=stream))

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [step(s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(p, q) for p, q in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, want))


def test_refusals(tsx):
    x, _ = values((4, 64), "bf16", 70)
    w = dev(np.ones(64))

    def refused(f, code=None):
        with pytest.raises(tsx.TsxError) as e:
            f()
        assert code is None or e.value.code == code
        assert len(str(e.value)) > 15

    for make in (lambda: tsx.Packer("f64", 4, 64), lambda: tsx.Packer("bf16", 4, 64, block=48),
                 lambda: tsx.Packer("bf16", 4, 64, form="int4"), lambda: tsx.GatedAct("bf16", 4, 64, act="relu"),
                 lambda: tsx.GroupNorm("bf16", 1, 4, 64, 7), lambda: tsx.GroupNorm("bf16", 1, 4, 64, 0),
                 lambda: tsx.GroupNorm("bf16", 1, 4, 64, 8, eps=-1.0),
                 lambda: tsx.GroupNorm("bf16", 1, 4, 64, 8, param_dtype="f16"),
                 lambda: tsx.GroupNorm("bf16", 1, 4, 64, 8, x_pitch=63),
                 lambda: tsx.GroupNorm("bf16", 1 << 20, 1 << 20, 64, 8)):
        refused(make, tsx.TSX_ERR_INVALID)
    pack = tsx.Packer("bf16", 4, 64)
    refused(lambda: pack.pack(x.float()), tsx.TSX_ERR_INVALID)
    refused(lambda: pack.pack(x.cpu()), tsx.TSX_ERR_INVALID)
    refused(lambda: pack.pack(x[:3]), tsx.TSX_ERR_INVALID)
    refused(lambda: pack.pack(x.t()), tsx.TSX_ERR_INVALID)
    refused(lambda: pack.unpack(tsx.Checkpoint(pack.pack(x).q, pack.pack(x).scale[:, :0])), tsx.TSX_ERR_INVALID)
    refused(lambda: tsx.Packer("bf16", 4, 64, pitch=63).pack(x), tsx.TSX_ERR_INVALID)
    glu = tsx.GatedAct("bf16", 4, 64)
    saved = pack.pack(x)
    refused(lambda: glu.backward(x, saved, x), tsx.TSX_ERR_INVALID)
    refused(lambda: glu.forward(x, x[:, :32]), tsx.TSX_ERR_INVALID)
    norm = tsx.GroupNorm("bf16", 1, 4, 64, 8)
    v = x.view(1, 4, 64)
    refused(lambda: norm.forward(v, w.bfloat16(), w), tsx.TSX_ERR_INVALID)
    refused(lambda: norm.forward(v, w[:32], w), tsx.TSX_ERR_INVALID)
    refused(lambda: norm.backward(v, v, w, w, w[:4], w[:8]), tsx.TSX_ERR_INVALID)
    # through the C names
    p, s = x.data_ptr(), torch.cuda.current_stream().cuda_stream
    head = (1, 4, 64, 64, 0, 128)
    assert tsx.tsx_pack(*head, p, None, p, s) == tsx.TSX_ERR_INVALID
    assert tsx.tsx_pack(*head, p + 1, p, p, s) == tsx.TSX_ERR_ALIGN
    assert "aligned" in tsx.tsx_last_error()
    assert tsx.tsx_pack(1, 0, 64, 64, 0, 128, None, None, None, s) == tsx.TSX_OK
    import ctypes
    d = tsx.tsx_norm_desc(1, 2, 0, 8, 0, 128, 1, 4, 64, 64, 64, 1e-5)
    ref_d = ctypes.byref(d)
    stats = torch.zeros(32, device="cuda")
    m = stats.data_ptr()
    small = tsx.tsx_group_norm_backward(ref_d, p, p, None, None, w.data_ptr(), w.data_ptr(), m, m, p, m, m, m, 8, s)
    assert small == tsx.TSX_ERR_INVALID and "workspace" in tsx.tsx_last_error()
    both = tsx.tsx_group_norm_backward(ref_d, p, p, p, m, w.data_ptr(), w.data_ptr(), m, m, p, m, m, m, 1 << 20, s)
    assert both == tsx.TSX_ERR_INVALID
