"""The operators of a feed-forward block and of a training step
(bitlinear_ffn.h) on the GPU, against plain float64 forms
(oracle/ffn_oracle.py).

What a definition rounds is compared bit for bit; sums are held to bounds by
arithmetic: U = 2^-24 is half a step of fp32, a result rounded to bf16 is off by
2^-8 of itself (half a step, relative), and the matrix cores' fp32 sums count a
whole step (2^-23) per term, as their rounding mode is not ours to choose.
"""

import weakref

import numpy as np
import pytest
import torch

import oracle
from oracle import ffn as ref
from oracle import layer

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
BF = 2.0 ** -8
TINY = 2.0 ** -126  # the smallest normal number of fp32 and bf16


@pytest.fixture(scope="module")
def bl():
    from bit_gemm_bitlinear_amd import bitlinear

    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return bitlinear


@pytest.fixture(scope="module")
def tr():
    from bit_gemm_bitlinear_amd import training

    return training


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def to_dev(bits):
    return dev(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16)


def bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def f64(t):
    return t.detach().double().cpu().numpy()


def bf16(a):
    """fp32 values of a rounded to bf16."""
    return oracle.bf16_to_f32(oracle.f32_to_bf16(np.asarray(a, np.float32)))


def codes(rng, m, k):
    """int8 codes (the whole range, -128 among them) and scales (one of a tiny
    row); every fifth row is zeros."""
    q = rng.integers(-128, 128, (m, k)).astype(np.int8)
    q[3::5] = 0
    s = np.exp(rng.standard_normal(m)).astype(np.float32) * 20
    s[1::7] = 1.27e7
    return q, s


def ternary(rng, n, k):
    """Ternary weights with whole zero rows, their packed form's bits and scale."""
    u = rng.integers(-1, 2, (n, k)).astype(np.int8)
    u[2::11] = 0
    return u, oracle.pack(u), np.float32(rng.uniform(20, 90))


def guarded(shape, dtype):
    """A tensor in the middle of a larger one filled with a pattern, and a check
    that the rest is as it was."""
    n = int(np.prod(shape))
    pad = 256
    whole = torch.full((n + 2 * pad,), 7, dtype=dtype, device=DEV)
    inner = whole[pad:pad + n].view(shape)

    def check():
        assert bool((whole[:pad] == 7).all()) and bool((whole[pad + n:] == 7).all()), "written outside the output"

    return inner, check


# ----------------------------------------------------------------- gated

SHAPES = [(1, 16, 256), (1, 1, 4), (2, 17, 260), (5, 40, 2084), (16, 33, 512), (17, 100, 1028), (31, 259, 252),
          (64, 130, 640), (77, 1003, 2084), (129, 300, 1280), (257, 515, 388), (300, 64, 4096), (1, 6912, 2560),
          (4, 4096, 1024), (513, 1024, 128), (16, 40, 6016),
          (9, 70, 9500), (3, 4200, 64), (17, 33, 128), (17, 33, 8192), (33, 8200, 8192), (100, 8200, 516), (257, 8200, 8192),
          (4104, 1001, 260), (1637, 1191, 13232), (19, 33, 4180), (2347, 782, 4), (1705, 33, 12604), (1956, 2155, 16),
          (1474, 14156, 4), (4284, 387, 12628), (21, 35, 12400), (27, 30, 5020), (3103, 35, 6768)]


def gated_inputs(bl, seed, m, n, k, tiled=False):
    rng = np.random.default_rng(seed)
    q, xs = codes(rng, m, k)
    (ug, pg, sg), (uu, pu, su) = ternary(rng, n, k), ternary(rng, n, k)
    tg, tu, dsg, dsu = dev(pg), dev(pu), dev(np.array([sg])), dev(np.array([su]))
    return q, xs, ug, sg, uu, su, tg, dsg, tu, dsu


def check_gated(a, g, u, want_a, act):
    """a against its float64 form.  g and u of that form are the kernel's own
    fp32 values.  relu2: three products, 3 U; silu: exp2's argument is rounded
    (|g| log2(e) at 2 U, times ln 2: 2 |g| U of e), exp2, the sum, the reciprocal
    and three products a step (2 U) each at most; the rounding to bf16.  exp2
    gives no value below the normal range but 0: exp(-|g|) is then off by TINY at
    most, and a = g u exp(-|g|) / (1 + exp(-|g|)) by |g u| TINY."""
    rel = 3 * U if act == "relu2" else (14 + 2 * np.abs(g.astype(np.float64))) * U
    tol = np.abs(want_a) * (BF * (1 + rel) + rel) + TINY
    if act == "silu":
        tol = tol + np.abs(g.astype(np.float64) * u) * TINY
    assert np.all(np.abs(a - want_a) <= tol), np.max(np.abs(a - want_a) / np.maximum(tol, 1e-300))


@pytest.mark.parametrize("act", ["relu2", "silu"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gated(bl, m, n, k, act):
    q, xs, ug, sg, uu, su, tg, dsg, tu, dsu = gated_inputs(bl, 11, m, n, k)
    w = bl.gated_weights(tg, dsg, tu, dsu)
    if n * k < 20000:
        assert np.array_equal(w.codes.flatten().cpu().numpy(), ref.gated_pack(ug, uu))
    outs, checks = zip(*(guarded((m, n), torch.bfloat16) for _ in range(3)))
    dq, dxs = dev(q), dev(xs)
    r = bl.GatedCall(dq, dxs, w, act, keep=True, out=bl.Gated(*outs))()
    for c in checks:
        c()
    want_a, g, u = ref.gated_forward(q, xs, ug, sg, uu, su, act)
    assert np.array_equal(bits_of(r.g), oracle.f32_to_bf16(g)) and np.array_equal(bits_of(r.u), oracle.f32_to_bf16(u))
    check_gated(f64(r.a), g, u, want_a, act)
    alone = bl.forward_gated(dq, dxs, w, act)
    assert alone.g is None and torch.equal(alone.a.view(torch.int16), r.a.view(torch.int16))


def test_gated_layouts_and_projections(bl):
    """Either layout of the packed weights, and g and u of the BitLinear calls."""
    m, n, k = 40, 96, 768
    q, xs, ug, sg, uu, su, tg, dsg, tu, dsu = gated_inputs(bl, 12, m, n, k)
    q = np.maximum(q, -127)  # codes as the quantizer writes them
    dq, dxs = dev(q), dev(xs)
    w = bl.gated_weights(tg, dsg, tu, dsu)
    for pg in (tg, bl.tile_weights(tg)):
        for pu in (tu, bl.tile_weights(tu)):
            assert torch.equal(bl.gated_weights(pg, dsg, pu, dsu, k=k).codes, w.codes)
    r = bl.forward_gated(dq, dxs, w, "silu", keep=True)
    ys = bl.GroupedQuantizedCall([dq] * 2, [dxs] * 2, [tg, tu], [dsg, dsu])()
    assert torch.equal(r.g, ys[0]) and torch.equal(r.u, ys[1])


@pytest.mark.parametrize("act", ["relu2", "silu"])
def test_gated_extremes(bl, act):
    """Projections far outside silu's and relu2's ordinary range, from scales."""
    m, n, k = 20, 48, 256
    q, xs, ug, sg, uu, su, tg, _, tu, _ = gated_inputs(bl, 13, m, n, k)
    xs[:] = 1.0
    for gs, us in ((1e-6, 1e-9), (1e6, 1.0), (1e-2, 1e12), (1e12, 1e-12), (3e-17, 1e3)):
        gs, us = np.float32(gs), np.float32(us)
        r = bl.forward_gated(dev(q), dev(xs), bl.gated_weights(tg, dev(np.array([gs])), tu, dev(np.array([us]))), act,
                             keep=True)
        with np.errstate(over="ignore"):
            want_a, g, u = ref.gated_forward(q, xs, ug, gs, uu, us, act)
        a = f64(r.a)
        fine = np.abs(want_a) < 3e38
        if act == "relu2":
            assert np.all(np.isfinite(a[fine]))
            # r * u may be below the normal range where the result is not
            fine &= (np.abs(g.astype(np.float64) * u) > TINY) | (g <= 0) | (u == 0)
        check_gated(a[fine], g[fine], u[fine], want_a[fine], act)


def test_gated_one_bad_row(bl):
    """A scale that is not finite spoils its row and no other."""
    for m in (3, 40):
        q, xs, ug, sg, uu, su, tg, dsg, tu, dsu = gated_inputs(bl, 14, m, 64, 512)
        w = bl.gated_weights(tg, dsg, tu, dsu)
        good = bl.forward_gated(dev(q), dev(xs), w, "silu").a
        xs[1] = np.nan
        bad = bl.forward_gated(dev(q), dev(xs), w, "silu").a
        keep = [i for i in range(m) if i != 1]
        assert torch.equal(bad[keep], good[keep]) and not bool(torch.isfinite(bad[1]).any())


@pytest.mark.parametrize("act", ["relu2", "silu"])
@pytest.mark.parametrize("m,n,k", [(3, 64, 512), (40, 64, 512), (20, 48, 8192), (300, 200, 260)])
def test_gated_nan_row(bl, m, n, k, act):
    """A projection that is not a number does not become one by its activation."""
    q, xs, ug, sg, uu, su, tg, dsg, tu, dsu = gated_inputs(bl, 15, m, n, k)
    w = bl.gated_weights(tg, dsg, tu, dsu)
    good = bl.forward_gated(dev(q), dev(xs), w, act, keep=True)
    xs[1] = np.nan
    bad = bl.forward_gated(dev(q), dev(xs), w, act, keep=True)
    others = [i for i in range(m) if i != 1]
    for b, g in zip(bad, good):
        assert bool(torch.isnan(b[1]).all()) and torch.equal(b[others], g[others])


BACK = [(1, 1, 4), (1, 16, 64), (3, 5, 8), (64, 64, 64), (65, 67, 68), (40, 1000, 260), (301, 1001, 1284), (130, 520, 640),
        (700, 200, 520), (520, 2048, 516), (17, 515, 128), (100, 2050, 2080), (130, 33, 8192), (513, 515, 8192),
        (1025, 33, 128), (2048, 33, 2080), (2048, 2050, 128), (1030, 260, 2052),
        (1350, 36, 4), (1115, 2867, 80), (141, 2788, 5420), (73, 2434, 1036)]


def backward_inputs(bl, seed, m, n, k):
    rng = np.random.default_rng(seed)
    q, xs, ug, sg, uu, su, tg, dsg, tu, dsu = gated_inputs(bl, seed, m, n, k)
    da, g, u = (bf16(rng.standard_normal((m, n)) * s) for s in (1e-3, 1.5, 1.5))
    da[2::5] = 0
    g[:, ::13] = 0
    return q, xs, ug, sg, uu, su, tg, dsg, tu, dsu, da, g, u


def check_backward(out, want, m, n, res=None):
    dx, dwg, dwu = out
    if dx is not None:
        # 2 n terms; the ratio of the scales, the gate's sum times it and the
        # quotient: four more roundings; the rounding to bf16
        tol = want["dx_abs"] * ((2 * n + 4) * 2 * U) + TINY
        w = want["dx"] if res is None else want["dx"] + res
        tol = tol + BF * (np.abs(want["dx"]) + tol) + (0 if res is None else BF * (np.abs(w) + tol) * (1 + BF))
        assert np.all(np.abs(f64(dx) - w) <= tol), np.max(np.abs(f64(dx) - w) / tol)
    for got, name in ((dwg, "dw_gate"), (dwu, "dw_up")):
        if got is not None:
            tol = want[name + "_abs"] * ((m + 2) * 2 * U) + TINY
            assert np.all(np.abs(f64(got) - want[name]) <= tol), (name, np.max(np.abs(f64(got) - want[name]) / tol))


@pytest.mark.parametrize("act", ["relu2", "silu"])
@pytest.mark.parametrize("m,n,k", BACK)
def test_gated_backward(bl, m, n, k, act):
    q, xs, ug, sg, uu, su, tg, dsg, tu, dsu, da, g, u = backward_inputs(bl, 21, m, n, k)
    xhat = oracle.bf16_to_f32(layer.restore_activations(q, xs))
    want = ref.gated_backward(*(t.astype(np.float64) for t in (da, g, u)), act, ug, sg, uu, su, xhat)
    dda, dg, du = (to_dev(oracle.f32_to_bf16(t)) for t in (da, g, u))
    dx, ck0 = guarded((m, k), torch.bfloat16)
    dwg, ck1 = guarded((n, k), torch.float32)
    dwu, ck2 = guarded((n, k), torch.float32)
    call = bl.GatedBackwardCall(dda, dg, du, act, dev(q), dev(xs), tg, dsg, tu, dsu, dx=dx, dw_gate=dwg, dw_up=dwu)
    check_backward(call(), want, m, n)
    for c in (ck0, ck1, ck2):
        c()
    first = [t.clone() for t in call._out]
    for a, b in zip(first, call()):
        assert torch.equal(a, b)  # the same again
    # either part alone, and added to what is there
    alone = bl.GatedBackwardCall(dda, dg, du, act, gate=tg, gate_scale=dsg, up=tu, up_scale=dsu)()
    check_backward(alone, want, m, n)
    assert alone[1] is None and alone[2] is None
    alone = bl.GatedBackwardCall(dda, dg, du, act, dev(q), dev(xs))()
    check_backward(alone, want, m, n)
    assert alone[0] is None
    rng = np.random.default_rng(22)
    res = bf16(rng.standard_normal((m, k)) * 1e-3)
    dx = to_dev(oracle.f32_to_bf16(res))
    had = [torch.randn(n, k, device=DEV) for _ in range(2)]
    acc = [t.clone() for t in had]
    out = bl.GatedBackwardCall(dda, dg, du, act, dev(q), dev(xs), tg, dsg, tu, dsu, residual=dx, dx=dx, dw_gate=acc[0],
                               dw_up=acc[1], accumulate=True)()
    check_backward((out[0], None, None), want, m, n, res.astype(np.float64))
    for got, was, name in ((out[1], had[0], "dw_gate"), (out[2], had[1], "dw_up")):
        w = want[name] + f64(was)
        tol = want[name + "_abs"] * ((m + 2) * 2 * U) + U * np.abs(w) * 2 + TINY
        assert np.all(np.abs(f64(got) - w) <= tol), name


@pytest.mark.parametrize("act", ["relu2", "silu"])
def test_gate_gradients_bit_for_bit(bl, act):
    """One token whose restored activation is 1 in column 0: dw[:, 0] is dg and
    du.  (silu's float64 forms may differ in their last bits: a value at a border
    of fp32, one in 2^28, would be seen here.)"""
    n = 6000
    rng = np.random.default_rng(23)
    g = np.concatenate([rng.standard_normal(n - 20) * 4, [0, -0.0, 1e-30, -1e-30, 50, -50, 88, -88, 89, -89, 100, -100, 500,
                                                          -500, 1e4, -1e4, 1.2785, -1.2785, 3e-39, 1e-10]])
    g, da, u = bf16(g)[None], bf16(rng.standard_normal(n))[None], bf16(rng.standard_normal(n))[None]
    q = np.zeros((1, 4), np.int8)
    q[0, 0] = 127
    out = bl.GatedBackwardCall(*(to_dev(oracle.f32_to_bf16(t)) for t in (da, g, u)), act, dev(q),
                               dev(np.array([127], np.float32)))()
    dg, du = ref.gate_gradients(*(t.astype(np.float64) for t in (da, g, u)), act)
    for got, want in ((out[1], dg[0]), (out[2], du[0])):
        got = f64(got)[:, 0]
        same = (got == want) | (np.abs(want) < TINY)  # below the normal range the matrix cores may flush
        assert np.all(same), (got[~same], want[~same])
        assert not np.any(f64(out[1])[:, 1:])


@pytest.mark.parametrize("act", ["relu2", "silu"])
def test_gate_gradients_over_the_whole_range(bl, act):
    """As above, for magnitudes whose partial products leave fp32's range where
    the gradients do not."""
    n = 20000
    rng = np.random.default_rng(25)
    da, g, u = (bf16(np.ldexp(rng.uniform(1, 2, n) * rng.choice([-1, 1], n), rng.integers(-120, 120, n)))
                for _ in range(3))
    with np.errstate(over="ignore"):
        dg, du = ref.gate_gradients(*(t.astype(np.float64) for t in (da, g, u)), act)
    ok = [(np.abs(t) > TINY) & (np.abs(t) < 2.0 ** 127) for t in (dg, du)]
    part = np.abs(da.astype(np.float64) * u)
    assert min(t.sum() for t in ok) > 1000
    # (silu's derivative is of middle size or leaves the range itself)
    assert act == "silu" or (ok[0] & ((part < TINY) | (part > 2.0 ** 128))).sum() > 100
    q = np.zeros((1, 4), np.int8)
    q[0, 0] = 127
    out = bl.GatedBackwardCall(*(to_dev(oracle.f32_to_bf16(t[None])) for t in (da, g, u)), act, dev(q),
                               dev(np.array([127], np.float32)))()
    for got, want, o in ((out[1], dg, ok[0]), (out[2], du, ok[1])):
        assert np.array_equal(f64(got)[o, 0], want[o])


@pytest.mark.parametrize("act", ["relu2", "silu"])
@pytest.mark.parametrize("m,n,k", [(40, 70, 260), (300, 520, 516)])
def test_gated_backward_nan(bl, m, n, k, act):
    """One gate value that is not a number spoils its token's dx and its output's
    weight gradients, whole, and nothing else."""
    q, xs, ug, sg, uu, su, tg, dsg, tu, dsu, da, g, u = backward_inputs(bl, 26, m, n, k)
    da[1, 5] = 0.5
    args = [to_dev(oracle.f32_to_bf16(t)) for t in (da, g, u)]
    kw = dict(q=dev(q), x_scale=dev(xs), gate=tg, gate_scale=dsg, up=tu, up_scale=dsu)
    good = bl.GatedBackwardCall(*args, act, **kw)()
    args[1][1, 5] = float("nan")
    bad = bl.GatedBackwardCall(*args, act, **kw)()
    for b, w, at in ((bad[0], good[0], 1), (bad[1], good[1], 5), (bad[2], good[2], 5)):
        others = [i for i in range(len(w)) if i != at]
        assert bool(torch.isnan(b[at]).all()) and torch.equal(b[others], w[others])


def test_gated_backward_tiled_weights(bl):
    m, n, k = 70, 96, 512
    q, xs, ug, sg, uu, su, tg, dsg, tu, dsu, da, g, u = backward_inputs(bl, 24, m, n, k)
    dda, dg, du = (to_dev(oracle.f32_to_bf16(t)) for t in (da, g, u))
    want = bl.GatedBackwardCall(dda, dg, du, "silu", gate=tg, gate_scale=dsg, up=tu, up_scale=dsu)()[0]
    for pg in (tg, bl.tile_weights(tg)):
        for pu in (tu, bl.tile_weights(tu)):
            got = bl.GatedBackwardCall(dda, dg, du, "silu", gate=pg, gate_scale=dsg, up=pu, up_scale=dsu, k=k)()[0]
            assert torch.equal(got, want)


@pytest.mark.parametrize("act", ["relu2", "silu"])
def test_gated_backward_against_differences(bl, act):
    """The directional derivatives of <da, act(g) u> along the restored
    activations and along the (unrounded) weights, in float64, against the
    gradients: what g and u are rounded to (bf16) and dg and du cost at most 2^-8
    each of every term's magnitude, to which act'(g) answers with its own slope
    (2 at most for relu2 near 0 relative to itself, |g act''| for silu)."""
    m, n, k = 24, 40, 64
    q, xs, ug, sg, uu, su, tg, dsg, tu, dsu, da, _, _ = backward_inputs(bl, 25, m, n, k)
    rng = np.random.default_rng(26)
    xs[:] = 40.0
    xhat = oracle.bf16_to_f32(layer.restore_activations(q, xs)).astype(np.float64)
    wg, wu = ug / np.float64(sg) + 0, uu / np.float64(su) + 0
    g, u = bf16(xhat @ wg.T), bf16(xhat @ wu.T)
    out = bl.GatedBackwardCall(*(to_dev(oracle.f32_to_bf16(t)) for t in (da, g, u)), act, dev(q), dev(xs), tg, dsg, tu,
                               dsu)()

    def value(x, a, b):
        return np.sum(da * ref.activation(act, x @ a.T)[0] * (x @ b.T))

    t = 1e-5
    # the magnitudes that the roundings act on
    g64, u64 = xhat @ wg.T, xhat @ wu.T
    h, dh = ref.activation(act, g64)
    mag_g = np.abs(da) * (np.abs(u64) * (np.abs(dh) + np.abs(g64) * (2 if act == "relu2" else 1)))
    mag_u = np.abs(da) * (np.abs(h) + np.abs(g64 * dh))
    for which in range(3):
        d = rng.standard_normal(((m, k), (n, k), (n, k))[which])
        args = [xhat, wg, wu]
        up, down = list(args), list(args)
        up[which], down[which] = args[which] + t * d, args[which] - t * d
        num = (value(*up) - value(*down)) / (2 * t)
        got = np.sum(f64(out[which]) * d)
        if which == 0:
            mag = np.sum(mag_g * np.abs(d @ wg.T) + mag_u * np.abs(d @ wu.T)) + np.sum(np.abs(f64(out[0]) * d))
        else:
            mag = np.sum((mag_g, mag_u)[which - 1] * np.abs(xhat @ d.T))
        assert abs(got - num) <= 3 * BF * mag, (which, got, num, mag)


# -------------------------------------------------------------------- w8

W8_SHAPES = [(1, 1, 4), (1, 16, 64), (1, 4096, 1024), (2, 17, 68), (5, 40, 2084), (9, 1003, 2084), (16, 33, 512),
             (17, 100, 1028), (33, 64, 4096), (64, 130, 640), (77, 515, 388), (129, 300, 1280), (257, 259, 252),
             (300, 600, 2048), (600, 1030, 512), (3, 200, 16384), (16, 100, 14336), (12, 33, 9500), (2, 4200, 64),
             (17, 33, 128), (17, 33, 4096), (100, 4100, 8192), (130, 8200, 8192), (200, 8200, 260), (1025, 8200, 128),
             (72, 5851, 5360), (520, 4100, 516), (1030, 4101, 260), (76, 11238, 10264), (138, 11219, 13852),
             (157, 6253, 10824), (20, 37, 5172), (269, 13215, 16), (66, 2499, 16300), (260, 13997, 16), (309, 14354, 1928),
             (153, 5841, 7648), (141, 5525, 15108), (3236, 12715, 4)]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("m,n,k", W8_SHAPES)
def test_w8(bl, m, n, k, bias):
    rng = np.random.default_rng(31)
    q, xs = codes(rng, m, k)
    w = (0.02 * rng.standard_normal((n, k)) * np.exp(rng.standard_normal((n, 1)))).astype(np.float32)
    w[n // 2] = 0
    v, s = ref.w8_quant(w)
    packed = bl.pack_weights_w8(dev(w))
    assert np.array_equal(packed.codes.flatten().cpu().numpy(), ref.w8_pack(v))
    assert np.array_equal(packed.scale.cpu().numpy(), s)
    assert np.array_equal(bl.unpack_weights_w8(packed).cpu().numpy(), (v * s[:, None]).astype(np.float32))
    b = bf16(rng.standard_normal(n)) if bias else None
    want = ref.w8_forward(q, xs, v, s)
    if bias:
        want = oracle.add_bf16(want, np.broadcast_to(oracle.f32_to_bf16(b), want.shape))
    out, check = guarded((m, n), torch.bfloat16)
    call = bl.W8Call(dev(q), dev(xs), packed, out=out, bias=to_dev(oracle.f32_to_bf16(b)) if bias else None)
    for _ in range(2):
        assert np.array_equal(bits_of(call()), want)
    check()


def test_w8_extreme_weights(bl):
    """Rows of the smallest and largest magnitudes, and whole sums of the largest
    codes over the longest K."""
    w = np.zeros((5, 64), np.float32)
    w[0, 3], w[1, :], w[2, ::2], w[3, 7], w[4, :2] = 3e38, 1e-44, -1e-38, 1e-45, (1.0, -2.0)
    p = bl.pack_weights_w8(dev(w))
    v, s = ref.w8_quant(w)
    assert np.array_equal(p.scale.cpu().numpy(), s)
    assert np.array_equal(p.codes.flatten().cpu().numpy(), ref.w8_pack(v))
    for m in (1, 20):
        k = 2 ** 17
        q = torch.full((m, k), -128, dtype=torch.int8, device=DEV)
        wl = torch.ones(16, k, device=DEV)
        wl[1::2] *= -1
        y = bl.forward_w8(q, torch.full((m,), 128.0, device=DEV), bl.pack_weights_w8(wl))
        scale = np.float32(1) / np.float32(127)
        want = bf16([np.float32(np.float32(np.float32(-128 * 127 * k) * scale) / np.float32(128))])[0]
        assert bool((y[:, 0::2] == float(want)).all()) and bool((y[:, 1::2] == -float(want)).all())


# ------------------------------------------------------------------ clip

def gradient_set(rng, shapes, scale=1.0):
    """fp32 and bf16 gradients in turn: (device tensors, their fp32 values)."""
    out = []
    for i, s in enumerate(shapes):
        a = (rng.standard_normal(s) * scale).astype(np.float32)
        out.append(dev(a) if i % 2 == 0 else to_dev(oracle.f32_to_bf16(a)).view(s))
    return out, [t.float().cpu().numpy() for t in out]


def check_clip(norm, outs, vals, max_norm):
    """The factor is rounded to fp32 and so is its product with the gradient: off
    by (1 + U)^2 - 1 of itself, and by 1 + BF more in bf16 (2^-50: float64's part)."""
    want, c = ref.clip(vals, max_norm)
    assert abs(float(norm) - want) <= 2 * U * want + 1e-45
    for o, v in zip(outs, vals):
        w = v.astype(np.float64) * c
        tol = np.abs(w) * ((1 + U) ** 2 * (1 if o.dtype == torch.float32 else 1 + BF) - 1 + 2.0 ** -50) + TINY
        if c == 1.0:
            assert np.array_equal(o.float().cpu().numpy(), v)
        assert np.all(np.abs(f64(o) - w) <= tol)


CLIP_SETS = [[(1,)], [(3, 5), (7,)], [(0,), (5,), (0, 4)], [(1000, 333), (333,), (17, 5, 3), (4096, 64)],
             [(i % 37 + 1, 13) for i in range(250)], [(16384,), (16385,), (16383,), (1 << 20,), (5, 100003)]]


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9, float("inf")])
@pytest.mark.parametrize("shapes", CLIP_SETS, ids=range(len(CLIP_SETS)))
def test_clip(bl, shapes, max_norm):
    grads, vals = gradient_set(np.random.default_rng(41), shapes)
    assert abs(float(bl.grad_norm(grads)) - ref.clip(vals, 1.0)[0]) <= 2 * U * ref.clip(vals, 1.0)[0]
    outs = [torch.empty_like(g) for g in grads]
    call = bl.ClipGradsCall(grads, max_norm, outs=outs)
    for _ in range(2):
        norm, got = call()
        check_clip(norm, got, vals, max_norm)
    for g, v in zip(grads, vals):  # the gradients are as they were
        assert np.array_equal(g.float().cpu().numpy(), v)
    norm, got = bl.clip_grads(grads, max_norm)
    check_clip(norm, got, vals, max_norm)
    for g, o in zip(grads, outs):
        assert torch.equal(g, o)  # in place, the same bits


def test_clip_alignment_and_order(bl):
    """Tensors that start at any element and dense tensors of any order of
    dimensions; what lies beside them is left alone."""
    rng = np.random.default_rng(42)
    torch.manual_seed(42)
    grads, vals, checks = [], [], []
    for i, n in enumerate((5, 1000, 40001, 7, 16384 + 3)):
        for dtype in (torch.float32, torch.bfloat16):
            base = torch.full((n + 40,), 3.0, dtype=dtype, device=DEV)
            g = base[i + 1:i + 1 + n]
            g.copy_(torch.from_numpy(rng.standard_normal(n).astype(np.float32)))
            grads.append(g)
            checks.append((base, i + 1, n))
    t = torch.randn(60, 70, device=DEV)
    grads += [t.t(), torch.randn(3, 8, 5, 6, device=DEV).contiguous(memory_format=torch.channels_last)]
    vals = [g.float().cpu().numpy() for g in grads]
    norm, got = bl.clip_grads(grads, 0.7)
    check_clip(norm, got, vals, 0.7)
    for base, at, n in checks:
        assert bool((base[:at] == 3).all()) and bool((base[at + n:] == 3).all())
    with pytest.raises(ValueError):
        bl.clip_grads([torch.zeros(8, 8, device=DEV)[:, :4]], 1.0)
    with pytest.raises(TypeError):
        bl.clip_grads([torch.zeros(8, device=DEV, dtype=torch.float16)], 1.0)
    with pytest.raises(ValueError):
        bl.clip_grads([torch.zeros(8, 4, device=DEV)], 1.0, outs=[torch.zeros(4, 8, device=DEV)])
    with pytest.raises(bl.BitLinearError):  # the same gradient twice
        bl.clip_grads([t, t], 1.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("alike", [True, False])
def test_clip_views_of_one_buffer(bl, dtype, alike):
    """Gradients next to each other in one buffer, from any element on, and
    clipped ones that lie as they do or otherwise: every length around the
    kernels' pieces and chunks."""
    lens = list(range(1, 20)) + [2047, 2048, 2049, 2050, 2055, 4096, 4099, 70001, 65536, 1]
    total = sum(lens)
    torch.manual_seed(44)
    for at in (0, 1, 3, 7):
        src = torch.randn(total + 24, device=DEV).to(dtype)
        dst = torch.full_like(src, 3.0)
        grads = src[at:at + total].split(lens)
        shift = at if alike else at + 1
        outs = dst[shift:shift + total].split(lens)
        vals = [g.float().cpu().numpy() for g in grads]
        norm, got = bl.clip_grads(grads, 0.7, outs=outs)
        check_clip(norm, got, vals, 0.7)
        assert bool((dst[:shift] == 3).all()) and bool((dst[shift + total:] == 3).all())
        assert torch.equal(bl.grad_norm(grads), norm)
        kept = src.clone()
        norm, got = bl.clip_grads(grads, 0.7)
        check_clip(norm, got, vals, 0.7)
        assert torch.equal(src[:at], kept[:at]) and torch.equal(src[at + total:], kept[at + total:])


def test_clip_extremes(bl):
    """Magnitudes whose squares leave fp32, values that are not finite, zeros."""
    big = torch.full((1000,), 2e38, device=DEV)
    norm, (o,) = bl.clip_grads([big], 1.0, outs=[torch.empty_like(big)])
    assert float(norm) == float("inf")  # 6.3e39 in fp32
    c = np.float32(1 / (np.sqrt(1000 * float(np.float32(2e38)) ** 2) + 1e-6))
    assert c == 0 or np.all(np.abs(f64(o) - float(np.float32(2e38)) * float(c)) <= 4 * U * 0.04)
    small = torch.full((1000,), 1e-30, device=DEV)
    norm, (o,) = bl.clip_grads([small], 1e-31, outs=[torch.empty_like(small)])
    want = np.sqrt(1000) * float(np.float32(1e-30))
    assert abs(float(norm) - want) <= 2 * U * want
    assert np.all(np.abs(f64(o) - 1e-30 * 1e-31 / (want + 1e-6)) <= TINY)
    z = torch.zeros(77, device=DEV)
    norm, (o,) = bl.clip_grads([z], 0.0, outs=[torch.empty_like(z)])
    assert float(norm) == 0 and not bool(o.any())
    for bad in (float("nan"), float("inf"), -float("inf")):
        g = [torch.ones(100, device=DEV), torch.ones(50, device=DEV, dtype=torch.bfloat16)]
        g[0][7] = bad
        norm, o = bl.clip_grads(g, 1.0)
        if bad != bad:
            assert bool(torch.isnan(norm).all()) and all(bool(torch.isnan(t).all()) for t in o)
        else:
            assert float(norm) == float("inf")
            assert bool(torch.isnan(o[0][7])) and not bool(o[1].any()) and int(torch.count_nonzero(o[0])) == 1


def test_clip_grad_norm_of_a_module(tr):
    torch.manual_seed(43)
    ffn = tr.FeedForward(256, 512, device=DEV)
    x = torch.randn(30, 256, device=DEV).to(torch.bfloat16)
    _, y = ffn(x)
    y.float().square().sum().backward()
    params = list(ffn.parameters())
    want = [p.grad.clone() for p in params]
    total = float(torch.sqrt(sum(g.double().square().sum() for g in want)))
    norm = tr.clip_grad_norm(params + params[:1], 0.25 * total)  # a parameter listed twice counts once
    assert norm.dim() == 0 and abs(float(norm) - total) <= 2 * U * total
    for p, g in zip(params, want):
        assert torch.allclose(p.grad.double(), g.double() * (0.25 * total / (total + 1e-6)), rtol=4 * U, atol=0)


# ------------------------------------------------------------- together

def numpy_norm(h, rstd, w):
    return bf16((h * rstd[:, None]).astype(np.float32) * (1 if w is None else w))


@pytest.mark.parametrize("act", ["relu2", "silu"])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_gated(bl, tr, act, residual):
    """The block's entry and its gradients, from the formulas of its steps."""
    torch.manual_seed(51)
    m, n, k = 45, 200, 260
    x = torch.randn(5, 9, k, device=DEV).to(torch.bfloat16).requires_grad_()
    r = torch.randn(5, 9, k, device=DEV).to(torch.bfloat16).requires_grad_() if residual else None
    nw = (1 + 0.1 * torch.randn(k, device=DEV)).requires_grad_()
    wg, wu = ((0.05 * torch.randn(n, k, device=DEV)).requires_grad_() for _ in range(2))
    h, a = tr.norm_gated(x, wg, wu, nw, r, act, 1e-5)
    assert a.shape == (5, 9, n) and h.shape == x.shape
    da = (torch.randn(5, 9, n, device=DEV) * 1e-2).to(torch.bfloat16)
    dh = (torch.randn(5, 9, k, device=DEV) * 1e-2).to(torch.bfloat16)
    torch.autograd.backward([a, h], [da, dh]) if residual else a.backward(da)
    # the same steps by the library's calls, whose own tests hold them
    normed = bl.rms_norm_quant(x.detach().reshape(m, k), nw.detach(), None if r is None else r.detach().reshape(m, k), 1e-5)
    (pg, sg), (pu, su) = bl.pack_weights(wg.detach()), bl.pack_weights(wu.detach())
    out = bl.forward_gated(normed.q, normed.x_scale, bl.gated_weights(pg, sg, pu, su), act, keep=True)
    assert torch.equal(a.reshape(m, n), out.a) and torch.equal(h.reshape(m, k), normed.h)
    xhat = f64(bl.restore_activations(normed.q, normed.x_scale))
    want = ref.gated_backward(f64(da).reshape(m, n), f64(out.g), f64(out.u), act, f64(bl.unpack_weights(pg)), float(sg),
                              f64(bl.unpack_weights(pu)), float(su), xhat)
    check_backward((None, wg.grad, wu.grad), want, m, n)
    dn, _, _ = bl.GatedBackwardCall(da.reshape(m, n), out.g, out.u, act, gate=pg, gate_scale=sg, up=pu, up_scale=su)()
    check_backward((dn, None, None), want, m, n)
    dx, dweight = bl.rms_norm_quant_backward(dn, normed.h, normed.rstd, nw.detach(), dh.reshape(m, k) if residual else None)
    assert torch.equal(x.grad.reshape(m, k), dx) and torch.equal(nw.grad, dweight)
    if residual:
        assert torch.equal(r.grad, x.grad) and r.grad.data_ptr() != x.grad.data_ptr()


@pytest.mark.parametrize("sub_norm", [False, True])
def test_feed_forward_block(bl, tr, sub_norm):
    """A whole block forward and backward: what it gives is what its calls give,
    and every parameter gets a gradient."""
    torch.manual_seed(52)
    ffn = tr.FeedForward(256, 680, "silu", sub_norm=sub_norm, device=DEV)
    x, r = (torch.randn(2, 21, 256, device=DEV).to(torch.bfloat16) for _ in range(2))
    h, y = ffn(x, r)
    assert torch.equal(h, x + r) and y.shape == x.shape
    (y.float() * torch.randn_like(y.float())).sum().backward()
    for name, p in ffn.named_parameters():
        assert p.grad is not None and bool(torch.isfinite(p.grad).all()) and bool(p.grad.any()), name
    norm = tr.clip_grad_norm(ffn.parameters(), 1.0)
    after = torch.sqrt(sum(p.grad.double().square().sum() for p in ffn.parameters()))
    assert float(after) <= max(1.0, float(norm)) * (1 + 1e-6)
    with torch.no_grad():
        h2, y2 = ffn(x, r)
        normed = bl.rms_norm_quant(x.reshape(42, -1), ffn.norm, r.reshape(42, -1), ffn.eps)
        w = bl.gated_weights(*bl.pack_weights(ffn.gate), *bl.pack_weights(ffn.up))
        a = bl.forward_gated(normed.q, normed.x_scale, w, "silu").a
        q, xs = (bl.rms_norm_quant(a, ffn.sub_norm, eps=ffn.eps)[:2] if sub_norm else bl.act_quant(a))
        want = bl.forward_quantized(q, xs, *bl.pack_weights(ffn.down))
    assert torch.equal(y2, y) and torch.equal(y2.reshape(42, -1), want) and torch.equal(h2, h)


def test_norm_gated_frozen_and_empty(tr):
    torch.manual_seed(53)
    n, k = 70, 128
    wg, wu = (0.05 * torch.randn(n, k, device=DEV) for _ in range(2))
    x = torch.randn(9, k, device=DEV).to(torch.bfloat16)
    for want in range(3):
        ts = [t.clone().requires_grad_(i == want) for i, t in enumerate((x, wg, wu))]
        _, a = tr.norm_gated(*ts)
        a.float().sum().backward()
        assert [t.grad is not None for t in ts] == [i == want for i in range(3)]
    _, a = tr.norm_gated(x, wg, wu)
    assert not a.requires_grad
    e = torch.zeros(0, 3, k, device=DEV, dtype=torch.bfloat16, requires_grad=True)
    w = wg.clone().requires_grad_()
    h, a = tr.norm_gated(e, w, wu, residual=e)
    assert a.shape == (0, 3, n) and h.shape == e.shape
    a.sum().backward()
    assert not bool(w.grad.any()) and w.grad.shape == w.shape
    # a not used: the gradient of h alone
    x2, r2 = x.clone().requires_grad_(), x.clone().requires_grad_()
    h, _ = tr.norm_gated(x2, w, wu, residual=r2)
    h.float().sum().backward()
    assert bool((x2.grad == 1).all()) and bool((r2.grad == 1).all())


def serving_calls(bl, m, seed=61):
    """A feed-forward block and an 8-bit head at m tokens, prepared."""
    torch.manual_seed(seed)
    k, n, v = 512, 1408, 1000
    x = torch.randn(m, k, device=DEV).to(torch.bfloat16)
    (pg, sg), (pu, su), (pd, sd) = (bl.pack_weights(0.05 * torch.randn(a, b, device=DEV)) for a, b in ((n, k), (n, k), (k, n)))
    head = bl.pack_weights_w8(0.05 * torch.randn(v, k, device=DEV))
    norm = bl.NormQuantCall(x)
    gated = bl.GatedCall(norm.out.q, norm.out.x_scale, bl.gated_weights(pg, sg, pu, su), "relu2")
    sub = bl.NormQuantCall(gated.out.a)
    down = bl.GroupedQuantizedCall([sub.out.q], [sub.out.x_scale], [pd], [sd], residuals=[x])
    last = bl.NormQuantCall(down.outs[0])
    logits = bl.W8Call(last.out.q, last.out.x_scale, head)
    calls = [norm, gated, sub, down, last, logits]
    return x, calls, logits.out


@pytest.mark.parametrize("m", [1, 4, 16, 17, 200])
def test_serving_block_in_a_graph(bl, m):
    """norm, gated projections, norm, down projection, norm, 8-bit head: captured,
    replayed with other tokens and eager work between, against eager runs."""
    x, calls, out = serving_calls(bl, m)
    x2, calls2, out2 = serving_calls(bl, m)
    for c in calls:
        c()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c in calls:
            c()
    for i in range(4):
        new = torch.randn(x.shape, device=DEV).to(torch.bfloat16)
        x.copy_(new)
        x2.copy_(new)
        out.zero_()
        graph.replay()
        for c in calls2:
            c()
        torch.cuda.synchronize()
        assert torch.equal(out, out2), i


def test_training_step_in_a_graph(bl, tr):
    """Forward, backward and clipping, captured and replayed."""
    m, n, k = 33, 300, 256
    rng = np.random.default_rng(62)
    q, xs, ug, sg, uu, su, tg, dsg, tu, dsu, da, g, u = backward_inputs(bl, 62, m, n, k)
    w = bl.gated_weights(tg, dsg, tu, dsu)
    dda = to_dev(oracle.f32_to_bf16(da))
    dq, dxs = dev(q), dev(xs)
    fwd = bl.GatedCall(dq, dxs, w, "silu", keep=True)
    back = bl.GatedBackwardCall(dda, fwd.out.g, fwd.out.u, "silu", dq, dxs, tg, dsg, tu, dsu)
    clip = bl.ClipGradsCall(list(back._out[1:]), 0.01)

    def step():
        fwd()
        back()
        return clip()

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        dda.copy_(to_dev(oracle.f32_to_bf16((rng.standard_normal((m, n)) * 1e-3).astype(np.float32))))
        dq.copy_(dev(codes(rng, m, k)[0]))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (fwd.out.a, *back._out, clip.norm)]
        f2 = bl.GatedCall(dq, dxs, w, "silu", keep=True)()
        b2 = bl.GatedBackwardCall(dda, f2.g, f2.u, "silu", dq, dxs, tg, dsg, tu, dsu)()
        norm, _ = bl.clip_grads(list(b2[1:]), 0.01)
        for a, b in zip(got, (f2.a, *b2, norm)):
            assert torch.equal(a, b)


def test_side_stream(bl):
    """Calls go to the current stream, in order with the work around them."""
    x, calls, out = serving_calls(bl, 24)
    for c in calls:
        c()
    want = out.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    new = x.clone()
    x.zero_()
    out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        x.copy_(new)
        for c in calls:
            c()
        got = out.clone()
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("act", ["relu2", "silu"])
def test_feed_forward_step_in_a_graph(bl, tr, act):
    """The module's forward and backward pass and the clipping of its gradients,
    captured once, against eager steps between the replays."""
    torch.manual_seed(63)
    m, k, n = 70, 256, 392
    ffn = tr.FeedForward(k, n, act, device=DEV)
    params = list(ffn.parameters())
    x = torch.randn(m, k, device=DEV).to(torch.bfloat16).requires_grad_()
    r = torch.randn(m, k, device=DEV).to(torch.bfloat16)
    dy = torch.randn(m, k, device=DEV).to(torch.bfloat16)

    def step():
        h, y = ffn(x, r)
        grads = torch.autograd.grad((y, h), (x, *params), (dy, r))
        norm, _ = bl.clip_grads(list(grads[1:]), 0.5)
        return (y.detach(), norm, *grads)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        with torch.no_grad():
            x.copy_(torch.randn(m, k, device=DEV))
            dy.copy_(torch.randn(m, k, device=DEV))
            for p in params:
                p.mul_(0.9)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i


def test_same_tensor_twice(bl, tr):
    """One weight as gate and up, one tensor as x and residual, g as u."""
    torch.manual_seed(64)
    m, n, k = 37, 130, 264
    x = torch.randn(m, k, device=DEV).to(torch.bfloat16).requires_grad_()
    w = (0.05 * torch.randn(n, k, device=DEV)).requires_grad_()
    w1, w2 = (w.detach().clone().requires_grad_() for _ in range(2))
    x1, x2 = (x.detach().clone().requires_grad_() for _ in range(2))
    da = torch.randn(m, n, device=DEV).to(torch.bfloat16)
    _, a = tr.norm_gated(x, w, w, residual=x, activation="silu")
    _, b = tr.norm_gated(x1, w1, w2, residual=x2, activation="silu")
    assert torch.equal(a, b)
    a.backward(da)
    b.backward(da)
    assert torch.equal(w.grad, w1.grad + w2.grad) and torch.equal(x.grad, x1.grad + x2.grad)
    (p, s), q, xs = bl.pack_weights(w.detach()), *bl.act_quant(x.detach())
    out = bl.forward_gated(q, xs, bl.gated_weights(p, s, p, s), "relu2", keep=True)
    assert torch.equal(out.g, out.u) and torch.equal(out.g, bl.forward_quantized(q, xs, p, s))
    one = bl.GatedBackwardCall(da, out.g, out.g, "relu2", q, xs, p, s, p, s)()
    two = bl.GatedBackwardCall(da, out.g, out.u, "relu2", q, xs, p, s, p, s)()
    assert all(torch.equal(i, j) for i, j in zip(one, two))


def test_broadcast_and_strided_inputs(bl, tr):
    """norm_gated of inputs that are not contiguous rows, against contiguous ones:
    a broadcast input's gradient is the sum over its copies."""
    torch.manual_seed(65)
    m, n, k = 24, 72, 256
    wg, wu = ((0.05 * torch.randn(n, k, device=DEV)).requires_grad_() for _ in range(2))
    da = torch.randn(n, m, device=DEV).to(torch.bfloat16).t()  # columns first
    one = torch.randn(1, k, device=DEV).to(torch.bfloat16).requires_grad_()
    wide = torch.randn(m, 2 * k, device=DEV).to(torch.bfloat16).requires_grad_()
    turned = torch.randn(k, m, device=DEV).to(torch.bfloat16).requires_grad_()
    for leaf, view in ((one, lambda t: t.expand(m, k)), (wide, lambda t: t[:, 1:2 * k:2]), (turned, lambda t: t.t())):
        for act in ("relu2", "silu"):
            rows = view(leaf).detach().contiguous().requires_grad_()
            got, want = tr.norm_gated(view(leaf), wg, wu, activation=act)[1], tr.norm_gated(rows, wg, wu, activation=act)[1]
            assert torch.equal(got, want)
            got = torch.autograd.grad(got, (leaf, wg, wu), da)
            want = torch.autograd.grad(want, (rows, wg, wu), da.contiguous())
            assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
            full = torch.autograd.grad(view(leaf), leaf, want[0])[0]  # what torch makes of the same rows
            assert torch.equal(got[0], full)


def test_calls_from_threads(bl):
    """Host threads with streams, shapes and workspaces of their own."""
    import threading

    def calls(i):
        q, xs, ug, sg, uu, su, tg, dsg, tu, dsu, da, g, u = backward_inputs(bl, 70 + i, 20 + 90 * i, 200 + 8 * i, 1024)
        dda, dg, du = (to_dev(oracle.f32_to_bf16(t)) for t in (da, g, u))
        dq, dxs = dev(q), dev(xs)
        w8 = bl.pack_weights_w8(torch.from_numpy(ug.astype(np.float32)).to(DEV))
        back = bl.GatedBackwardCall(dda, dg, du, "silu", dq, dxs, tg, dsg, tu, dsu)
        outs = [torch.empty_like(t) for t in back._out[1:]]
        return (bl.GatedCall(dq, dxs, bl.gated_weights(tg, dsg, tu, dsu), "silu"), bl.W8Call(dq, dxs, w8), back,
                bl.ClipGradsCall(list(back._out[1:]), 1e-3, outs=outs))

    def run(cs):
        for c in cs:
            c()
        return [cs[0].out.a, cs[1].out, *cs[2]._out, cs[3].norm, *cs[3].outs]

    sets = [calls(i) for i in range(4)]
    want = [[t.clone() for t in run(cs)] for cs in sets]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got = run(sets[i])
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    bad.append(i)
        except Exception as e:  # reported by the main thread
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


@pytest.mark.parametrize("m,n,k", [(2 ** 21, 1, 4), (1, 2 ** 20, 4), (3, 5, 2 ** 22), (40, 2 ** 20, 4)])
def test_gated_backward_largest_sizes(bl, m, n, k):
    q, xs, ug, sg, uu, su, tg, dsg, tu, dsu, da, g, u = backward_inputs(bl, 72, m, n, k)
    xhat = oracle.bf16_to_f32(layer.restore_activations(q, xs))
    want = ref.gated_backward(*(t.astype(np.float64) for t in (da, g, u)), "relu2", ug, sg, uu, su, xhat)
    args = [to_dev(oracle.f32_to_bf16(t)) for t in (da, g, u)]
    check_backward(bl.GatedBackwardCall(*args, "relu2", dev(q), dev(xs), tg, dsg, tu, dsu)(), want, m, n)


def test_refusals(bl):
    """What does not fit is refused before anything runs, and leaves outputs as
    they were."""
    m, n, k = 40, 48, 512
    q, xs, ug, sg, uu, su, tg, dsg, tu, dsu, da, g, u = backward_inputs(bl, 73, m, n, k)
    dq, dxs = dev(q), dev(xs)
    dda, dg, du = (to_dev(oracle.f32_to_bf16(t)) for t in (da, g, u))
    w, w8 = bl.gated_weights(tg, dsg, tu, dsu), bl.pack_weights_w8(torch.randn(n, k, device=DEV))
    out = torch.full((m, n), 3.0, dtype=torch.bfloat16, device=DEV)
    bad = (ValueError, TypeError, bl.BitLinearError)
    for call in (lambda: bl.forward_w8(dq[:, :256].contiguous(), dxs, w8, out=out),  # another width
                 lambda: bl.forward_w8(dq[:, ::2], dxs, w8, out=out),
                 lambda: bl.forward_w8(dq, dxs[:-1], w8, out=out),
                 lambda: bl.forward_w8(dq, dxs.double(), w8, out=out),
                 lambda: bl.forward_w8(dq, dxs, w8, out=out[:-1]),
                 lambda: bl.forward_w8(dq, dxs, w8, out=out, bias=torch.zeros(n, device=DEV)),
                 lambda: bl.forward_w8(dq, dxs, w8._replace(n=n + 16), out=out),
                 lambda: bl.forward_w8(dq, dxs, w8._replace(codes=w8.codes.cpu()), out=out),
                 lambda: bl.forward_w8(dq.cpu(), dxs, w8, out=out),
                 lambda: bl.forward_w8(dq, dxs, w8, out=out, bias=out.view(-1)[:n]),  # overlaps
                 lambda: bl.GatedCall(dq, dxs, w, "gelu", out=bl.Gated(out, None, None))(),
                 lambda: bl.GatedCall(dq, dxs, w, "silu", keep=True, out=bl.Gated(out, None, None))(),
                 lambda: bl.GatedCall(dq, dxs, w, "silu", out=bl.Gated(out, out, out))(),
                 lambda: bl.GatedCall(dq, dxs, w._replace(k=k - 256), "silu", out=bl.Gated(out, None, None))(),
                 lambda: bl.gated_weights(tg, dsg, tu[:32], dsu),
                 lambda: bl.gated_weights(tg, dsg, tu, dsu.double()),
                 lambda: bl.GatedBackwardCall(dda, dg, du, "silu"),
                 lambda: bl.GatedBackwardCall(dda, dg, du[:-1], "silu", dq, dxs),
                 lambda: bl.GatedBackwardCall(dda, dg, du, "silu", dq, dxs, tg, dsg),
                 lambda: bl.GatedBackwardCall(dda, dg, du, "silu", dq, dxs, accumulate=True),
                 lambda: bl.GatedBackwardCall(dda, dg, du, "silu", gate=tg, gate_scale=dsg, up=tu, up_scale=dsu,
                                              dx=dda.view(-1)[:0].view(0, k)),
                 lambda: bl.clip_grads([], 1.0),
                 lambda: bl.clip_grads([out, out[1:]], 1.0),
                 lambda: bl.clip_grads([out], 1.0, outs=[out.view(-1)[1:].view(-1)]),
                 lambda: bl.clip_grads([out, torch.zeros(4)], 1.0),
                 lambda: bl.clip_grads([out[:, ::2]], 1.0),
                 lambda: bl.clip_grads([out], -1.0)):
        with pytest.raises(bad):
            call()
    for make in (lambda ws: bl.GatedBackwardCall(dda, dg, du, "silu", dq, dxs, workspace=ws),
                 lambda ws: bl.GradNormCall([out], workspace=ws)):
        need = make(None).workspace.numel()
        assert need > 0
        with pytest.raises(bad):
            make(torch.empty(need - 256, dtype=torch.uint8, device=DEV))()
    assert bool((out == 3).all())


# The limits: tokens, outputs, width.
LIMITS = [(2 ** 19, 17, 4), (2 ** 19, 1, 20), (1, 2 ** 24, 4), (17, 2 ** 24, 4), (2, 19, 2 ** 17), (40, 19, 2 ** 17),
          (300, 19, 2 ** 17 - 4)]


@pytest.mark.parametrize("m,n,k", LIMITS)
def test_largest_sizes(bl, m, n, k):
    rng = np.random.default_rng(71)
    q, xs = dev(rng.integers(-128, 128, (m, k)).astype(np.int8)), torch.rand(m, device=DEV) + 0.5
    ends = torch.tensor(sorted({0, m // 2, m - 1}), device=DEV)
    cols = torch.tensor(sorted({0, n // 2, n - 1}), device=DEV)
    w = torch.randn(n, k, device=DEV)
    w8 = bl.pack_weights_w8(w)
    v = torch.round(bl.unpack_weights_w8(w8)[cols].double() / w8.scale[cols].double()[:, None])
    acc = (q[ends].double()[:, None, :] * v[None]).sum(-1).float()  # whole numbers under 2^53, rounded once
    y = bl.forward_w8(q, xs, w8)
    assert torch.equal(y[ends][:, cols], (acc * w8.scale[cols] / xs[ends][:, None]).to(torch.bfloat16))
    del y, w8
    packed, scale = bl.pack_weights(w)
    del w
    out = bl.forward_gated(q, xs, bl.gated_weights(packed, scale, packed, scale), "relu2", keep=True)
    u = torch.round(bl.unpack_weights(packed)[cols].double())
    acc = (q[ends].double()[:, None, :] * u[None]).sum(-1).float()
    g = acc / (xs[ends][:, None] * scale)
    assert torch.equal(out.g[ends][:, cols], g.to(torch.bfloat16)) and torch.equal(out.g, out.u)
    a, want = out.a[ends][:, cols].double(), g.double().relu() ** 2 * g.double()
    assert bool(((a - want).abs() <= want.abs() * (BF * (1 + 3 * U) + 3 * U) + TINY).all())


def test_large_offsets(bl):
    """Outputs and weights of more than 2^31 elements, and gradients too."""
    m, n, k = 70000, 32768, 64
    q = torch.randint(-127, 128, (m, k), device=DEV, dtype=torch.int8)
    xs = torch.full((m,), 50.0, device=DEV)
    w = 0.05 * torch.randn(n, k, device=DEV)
    p = bl.pack_weights_w8(w)
    y = bl.forward_w8(q, xs, p)
    rows = [0, 1, 32767, 65535, 65536, m - 1]
    assert torch.equal(y[rows], bl.forward_w8(q[rows].contiguous(), xs[:6].contiguous(), p))
    del y
    (pg, sg), (pu, su) = bl.pack_weights(w), bl.pack_weights(w.flip(0).contiguous())
    gw = bl.gated_weights(pg, sg, pu, su)
    a = bl.forward_gated(q, xs, gw, "relu2").a
    assert torch.equal(a[rows], bl.forward_gated(q[rows].contiguous(), xs[:6].contiguous(), gw, "relu2").a)
    del a
    g = torch.zeros(2 ** 31 + 5, device=DEV, dtype=torch.bfloat16)
    g[-1], g[2 ** 31], g[0] = 3.0, 4.0, 12.0
    norm, (o,) = bl.clip_grads([g], 6.5)
    assert float(norm) == 13.0
    assert [float(o[i]) for i in (0, 2 ** 31, 2 ** 31 + 4)] == [6.0, 2.0, 1.5]
    del g, o
    n, k = 32768, 65536 + 256
    codes_ = torch.zeros(n // 16, k // 64, 4, 16, 16, dtype=torch.int8, device=DEV)
    codes_[-1, -1, 3, 15, 15] = 5  # weight [n - 1][k - 1]
    codes_[0, 0, 0, 0, 0] = 7
    w8 = bl.W8Weights(codes_, torch.ones(n, device=DEV), n, k)
    q = torch.full((1, k), 2, device=DEV, dtype=torch.int8)
    y = bl.forward_w8(q, torch.ones(1, device=DEV), w8)
    assert float(y[0, -1]) == 10 and float(y[0, 0]) == 14 and int(torch.count_nonzero(y)) == 2


def test_odd_width_past_four_gigabytes_of_codes(bl):
    """Tiles that load activations in words, of a product whose codes are more than
    2^32 bytes: every row against the same rows in calls of their own."""
    m, n, k = 65552, 64, 65540
    gen = torch.Generator(device=DEV).manual_seed(75)
    q = torch.empty((m, k), dtype=torch.int8, device=DEV)
    for i in range(0, m, 8192):
        q[i:i + 8192] = torch.randint(-128, 128, q[i:i + 8192].shape, generator=gen, device=DEV, dtype=torch.int8)
    xs = torch.rand(m, generator=gen, device=DEV) + 0.5
    w = torch.randn(n, k, generator=gen, device=DEV)
    w8 = bl.pack_weights_w8(w)
    packed, scale = bl.pack_weights(w)
    gw = bl.gated_weights(packed, scale, packed.flip(0).contiguous(), scale)
    y, a = bl.forward_w8(q, xs, w8), bl.forward_gated(q, xs, gw, "relu2", keep=True)
    for i in list(range(0, 512, 128)) + [m // 2, m - 128]:  # the first rows are the farthest from the end
        part, ps = q[i:i + 128].clone(), xs[i:i + 128].clone()
        assert torch.equal(y[i:i + 128], bl.forward_w8(part, ps, w8)), i
        small = bl.forward_gated(part, ps, gw, "relu2", keep=True)
        assert all(torch.equal(b[i:i + 128], c) for b, c in zip(a, small)), i


@pytest.mark.parametrize("gs,us", [(1e-17, 1e-17), (10, 1e-34), (20, 1e-34), (1e-30, 1e5)])
@pytest.mark.parametrize("m,n,k", [(3, 64, 512), (40, 64, 512), (20, 48, 8192), (300, 200, 260)])
def test_gated_silu_of_large_factors(bl, m, n, k, gs, us):
    """Projections that are both large: no step leaves fp32's range where the result
    does not.  Within |g| < 88 as check_gated has it; above, the sigmoid of g >= 0 is 1 to
    2^-126, and the rest is two products and the rounding to bf16; below, the
    result is |g u| exp(-88) at most, and exp(-88) is under TINY."""
    q, xs, ug, _, uu, _, tg, _, tu, _ = gated_inputs(bl, 16, m, n, k)
    xs[:] = 1.0
    gs, us = np.float32(gs), np.float32(us)
    r = bl.forward_gated(dev(q), dev(xs), bl.gated_weights(tg, dev(np.array([gs])), tu, dev(np.array([us]))), "silu",
                         keep=True)
    want, g, u = ref.gated_forward(q, xs, ug, gs, uu, us, "silu")
    a, gu = f64(r.a), g.astype(np.float64) * u
    assert np.isfinite(g).all() and np.isfinite(u).all()
    assert us > 1 or np.abs(gu[g < 0]).max() > 3.5e38  # g * u alone leaves the range
    assert not np.isnan(a).any()
    fine = np.abs(want) < 3.3e38
    assert np.isfinite(a[fine]).all()
    over = np.abs(want) > 3.41e38  # past bf16's largest value and half a step
    assert np.array_equal(a[over], np.sign(want[over]) * np.inf)
    mid = fine & (np.abs(g) < 88)
    check_gated(a[mid], g[mid], u[mid], want[mid], "silu")
    high = fine & (g >= 88)
    assert np.all(np.abs(a - gu)[high] <= np.abs(gu[high]) * (BF * (1 + 6 * U) + 6 * U) + TINY)
    low = fine & (g <= -88)
    assert np.all(np.abs(a[low]) <= np.abs(gu[low]) * TINY)


@pytest.mark.parametrize("m", [1, 9, 40, 300])
@pytest.mark.parametrize("k", [64, 68, 4096])
def test_w8_weights_that_are_not_finite(bl, m, k):
    """A weight that is not a number, or infinite, spoils its row's scale and all of that
    output's values, and no others."""
    torch.manual_seed(76)
    n = 70
    q, xs = (dev(t) for t in codes(np.random.default_rng(76), m, k))
    w = 0.02 * torch.randn(n, k, device=DEV)
    good = bl.pack_weights_w8(w)
    y = bl.forward_w8(q, xs, good)
    nan, inf = float("nan"), float("inf")
    for values, kind in (((nan,), torch.isnan), ((inf,), torch.isinf), ((-inf, 1.0), torch.isinf), ((inf, nan), torch.isnan),
                         ((-nan, -inf), torch.isnan)):
        for at in (0, k - len(values), min(k - 4, 63)):
            bad = w.clone()
            bad[33, at:at + len(values)] = torch.tensor(values, device=DEV)
            p = bl.pack_weights_w8(bad)
            others = [i for i in range(n) if i != 33]
            assert bool(kind(p.scale[33])) and torch.equal(p.scale[others], good.scale[others])
            got = bl.forward_w8(q, xs, p)
            assert not bool(torch.isfinite(got[:, 33]).any())
            assert torch.equal(got[:, others], y[:, others])
            assert torch.equal(bl.unpack_weights_w8(p)[others], bl.unpack_weights_w8(good)[others])


def test_gradients_from_a_generator(bl):
    """Prepared calls hold the tensors that a generator made for them."""
    torch.manual_seed(77)
    src = [torch.randn(5000 + i, device=DEV).to(torch.bfloat16) for i in range(20)]
    total = float(torch.sqrt(sum(t.double().square().sum() for t in src)))
    for make in (bl.GradNormCall, lambda it: bl.ClipGradsCall(it, 0.5)):
        refs = []

        def made():
            for t in src:
                g = t.float()
                refs.append(weakref.ref(g))
                yield g
                del g

        call = make(made())
        assert len(refs) == 20 and all(r() is not None for r in refs)
        other = [torch.full((5000 + i,), 1e9, device=DEV) for i in range(20)]  # on what would be free
        norm = call()
        norm = norm[0] if isinstance(norm, tuple) else norm
        assert abs(float(norm) - total) <= 2 * U * total
        del other
    assert abs(float(bl.grad_norm(t.float() for t in src)) - total) <= 2 * U * total
    norm, outs = bl.clip_grads((t.float() for t in src), 0.5)
    assert abs(float(norm) - total) <= 2 * U * total
    for o, t in zip(outs, src):
        assert torch.allclose(o.double(), t.double() * (0.5 / (total + 1e-6)), rtol=4 * U, atol=0)


def test_clipping_is_seen_by_autograd(bl, tr):
    """Clipping in place a tensor that a graph has saved makes that graph's backward
    pass an error, as torch's own in-place operations do."""
    def saved(x):
        g = torch.autograd.grad(x.square().sum(), x, create_graph=True)[0]
        return g, g.square().sum()  # saves g

    x = torch.randn(50, device=DEV, requires_grad=True)
    for clip in (lambda g: bl.clip_grads([g], 0.1), lambda g: bl.clip_grads([g.detach()], 0.1),
                 lambda g: bl.clip_grads([torch.zeros_like(g)], 0.1, outs=[g])):
        g, loss = saved(x)
        clip(g)
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
    p = torch.nn.Parameter(x.detach().clone())
    g, loss = saved(p)
    p.grad = g
    tr.clip_grad_norm([p], 0.1)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    # what is only read stays usable
    g, loss = saved(x)
    want = torch.autograd.grad(loss, x, retain_graph=True)[0]
    bl.grad_norm([g])
    bl.clip_grads([g], 0.1, outs=[torch.empty_like(g)])
    assert torch.equal(torch.autograd.grad(loss, x)[0], want)
    with torch.inference_mode():  # tensors without a version
        g = torch.full((100,), 2.0, device=DEV)
        norm, (o,) = bl.clip_grads([g], 10.0)
    assert float(norm) == 20 and bool((o - 1).abs().max() < 1e-6)


def test_clip_grad_norm_without_a_gradient(tr):
    """Zero on the parameters' device, from any iterable."""
    ffn = tr.FeedForward(64, 128, device=DEV)
    want = torch.zeros((), device=DEV)
    for params in (ffn.parameters(), list(ffn.parameters()), ffn.gate, (p for p in ffn.parameters())):
        norm = tr.clip_grad_norm(params, 1.0)
        assert norm.device == want.device and norm.dtype == torch.float32 and norm.dim() == 0 and float(norm) == 0
    torch.stack([norm, want])
    assert float(tr.clip_grad_norm([], 1.0)) == 0
