"""The operators around the product (bitlinear_layer.h) on the GPU, against
plain float64 forms (oracle/layer_oracle.py).

What a definition rounds is compared bit for bit; sums are held to bounds by
arithmetic: u = 2^-24 is half a step of fp32, a sum of t terms in any order is
off by at most t steps of the sum of their magnitudes, and a result rounded to
bf16 by 2^-8 of itself (half a step, relative).  The matrix cores' fp32 sums
count a whole step (2^-23) per term, as their rounding mode is not ours to
choose.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import layer as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
BF = 2.0 ** -8


@pytest.fixture(scope="module")
def bl():
    from bit_gemm_bitlinear_amd import bitlinear

    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return bitlinear


def to_dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(DEV)


def bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def f64(t):
    return t.double().cpu().numpy()


def bf16_bits(a):
    return oracle.f32_to_bf16(np.asarray(a, np.float32))


def rows(rng, m, k, scale=1.0):
    """Rows with a few large channels; every fifth row is zero, and every
    seventh tiny (its codes' scale is clamped without a large weight)."""
    x = rng.standard_normal((m, k)) * scale
    x[:, rng.random(k) < 0.02] *= 20
    x[3::5] = 0
    x[6::7] *= 1e-9
    return bf16_bits(x)


def make_weight(rng, kind, k):
    if kind == "none":
        return None, None
    w = 1 + 0.2 * rng.standard_normal(k)
    if kind == "bf16":
        b = bf16_bits(w)
        return to_dev(b), oracle.bf16_to_f32(b)
    w = w.astype(np.float32)
    return torch.from_numpy(w).to(DEV), w


# ------------------------------------------------------------------ norm

NORM_SHAPES = [(1, 4), (1, 8), (3, 12), (9, 2048), (5, 2052), (8, 4096), (2, 6912), (7, 14332),
               (4, 16384), (3, 16388), (2, 20000), (300, 260)]


@pytest.mark.parametrize("weight", ["none", "bf16", "fp32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("m,k", NORM_SHAPES)
def test_norm_quant(bl, m, k, residual, weight):
    rng = np.random.default_rng([1, m, k, residual])
    x = rows(rng, m, k)
    r = rows(rng, m, k, 3.0) if residual else None
    wt, wf = make_weight(rng, weight, k)
    eps = 1e-5
    got = bl.rms_norm_quant(to_dev(x), wt, None if r is None else to_dev(r), eps=eps, want_norm=True)
    rstd = got.rstd.cpu().numpy()
    want = ref.rms_rstd(ref.residual_sum(x, r), eps)
    # fp64 sums are off by less than 2^-30: rstd is the rounded value or, at a
    # border, its neighbour
    assert np.all(np.abs(rstd - want) <= (U + 2.0 ** -30) * want)
    q, s, h, _, n = ref.rms_norm_quant(x, r, wf, eps, rstd=rstd)
    assert np.array_equal(bits_of(got.h), h)
    assert np.array_equal(bits_of(got.n), n)
    assert np.array_equal(got.x_scale.cpu().numpy(), s)
    assert np.array_equal(got.q.cpu().numpy(), q)
    # the fused codes are those of the separate call on the norm's output
    q2, s2 = bl.act_quant(got.n)
    assert torch.equal(q2, got.q) and torch.equal(s2, got.x_scale)


@pytest.mark.parametrize("k", [64, 4100, 9000, 16388])
def test_norm_not_finite_stays_in_its_row(bl, k):
    """A residual add that overflows, or a NaN: 1 / rms of 0 or NaN, and no
    other row's outputs or gradients change."""
    rng = np.random.default_rng([6, k])
    x, r = rows(rng, 9, k), rows(rng, 9, k)
    wt, _ = make_weight(rng, "bf16", k)
    dn, dh = to_dev(rows(rng, 9, k)), to_dev(rows(rng, 9, k))
    clean = bl.rms_norm_quant(to_dev(x), wt, to_dev(r), want_norm=True)
    cdx, _ = bl.rms_norm_quant_backward(dn, clean.h, clean.rstd, wt, dh)
    xt, rt = to_dev(x), to_dev(r)
    xt[2, k - 1] = rt[2, k - 1] = 3e38
    xt[5, 1] = float("nan")
    got = bl.rms_norm_quant(xt, wt, rt, want_norm=True)
    assert got.rstd[2] == 0 and bool(got.rstd[5].isnan())
    dx, _ = bl.rms_norm_quant_backward(dn, got.h, got.rstd, wt, dh)
    keep = [0, 1, 3, 4, 6, 7, 8]
    for a, c in zip((*got, dx), (*clean, cdx)):
        assert torch.equal(a[keep], c[keep])


@pytest.mark.parametrize("k", [64, 2052, 16388])
@pytest.mark.parametrize("which", ["x", "residual"])
def test_norm_quant_in_place(bl, k, which):
    rng = np.random.default_rng([2, k])
    x, r = rows(rng, 6, k), rows(rng, 6, k, 3.0)
    want = bl.rms_norm_quant(to_dev(x), None, to_dev(r))
    xt, rt = to_dev(x), to_dev(r)
    out = bl.Normed(torch.empty_like(want.q), torch.empty(6, device=DEV), xt if which == "x" else rt,
                    torch.empty(6, device=DEV), None)
    got = bl.NormQuantCall(xt, None, rt, out=out)()
    for a, b in zip(got[:4], want[:4]):
        assert torch.equal(a, b)


def test_norm_quant_leaves_other_rows(bl):
    """Rows behind the last token stay as they were."""
    rng = np.random.default_rng(3)
    x = to_dev(rows(rng, 5, 132))
    q = torch.full((8, 132), 77, dtype=torch.int8, device=DEV)
    s = torch.full((8,), 5.0, device=DEV)
    h = torch.full((8, 132), 3.0, dtype=torch.bfloat16, device=DEV)
    rstd = torch.full((8,), 6.0, device=DEV)
    bl.NormQuantCall(x, None, x.clone(), out=bl.Normed(q[:5], s[:5], h[:5], rstd[:5], None))()
    assert bool((q[5:] == 77).all()) and bool((s[5:] == 5).all())
    assert bool((h[5:] == 3).all()) and bool((rstd[5:] == 6).all())


def check_norm_backward(out, dxt, dwt, k, m, dh):
    # dx: the mean's k terms, two products and a subtraction in fp32, one
    # rounding to bf16
    inner = np.abs(out["r"] * out["g"]) + np.abs(out["r"] * out["z"]) * out["c_abs"]
    tol = BF * np.abs(out["dx"]) * (1 + BF) + (1 + BF) * U * (
        (k + 8) * np.abs(out["r"] * out["z"]) * out["c_abs"] + 6 * inner +
        (0 if dh is None else np.abs(dh)))
    assert np.all(np.abs(f64(dxt) - out["dx"]) <= tol + 1e-40)
    if dwt is not None:
        assert np.all(np.abs(f64(dwt) - out["dweight"]) <= (m + 4) * U * out["dw_abs"] + 1e-40)


@pytest.mark.parametrize("weight", ["none", "bf16", "fp32"])
@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("m,k", [(1, 4), (1, 2048), (3, 12), (8, 1032), (9, 1032), (8, 16388), (40, 2052), (9, 4096), (2, 14332), (3, 16384),
                                 (5, 16388), (1500, 64), (1100, 260), (1030, 16388)])
def test_norm_backward(bl, m, k, with_dh, weight):
    rng = np.random.default_rng([4, m, k])
    h = rows(rng, m, k)
    rstd = ref.rms_rstd(h, 1e-5).astype(np.float32)
    dn = bf16_bits(rng.standard_normal((m, k)) * 1e-3)
    dn[::4] = 0  # tokens that the loss masks out
    dh = bf16_bits(rng.standard_normal((m, k)) * 1e-3) if with_dh else None
    wt, wf = make_weight(rng, weight, k)
    dx, dw = bl.rms_norm_quant_backward(to_dev(dn), to_dev(h), torch.from_numpy(rstd).to(DEV), wt,
                                        None if dh is None else to_dev(dh))
    f = oracle.bf16_to_f32
    out = ref.rms_norm_quant_backward(f(dn), f(h), rstd, wf, None if dh is None else f(dh))
    check_norm_backward(out, dx, dw, k, m, None if dh is None else f(dh).astype(np.float64))
    assert (dw is None) == (weight == "none")


@pytest.mark.parametrize("m,k", [(37, 2056), (5, 2056), (8, 2056), (8, 8192), (7, 33000), (1, 33000)])
def test_norm_backward_in_place_and_accumulate(bl, m, k):
    rng = np.random.default_rng(5)
    h, dn, dh = rows(rng, m, k), bf16_bits(rng.standard_normal((m, k))), bf16_bits(rng.standard_normal((m, k)))
    rstd = torch.from_numpy(ref.rms_rstd(h, 1e-5).astype(np.float32)).to(DEV)
    wt, _ = make_weight(rng, "fp32", k)
    dx, dw = bl.rms_norm_quant_backward(to_dev(dn), to_dev(h), rstd, wt, to_dev(dh))
    for which in ("dn", "dh"):
        a, b = to_dev(dn), to_dev(dh)
        acc = torch.full((k,), 0.5, device=DEV)
        dx2, dw2 = bl.NormQuantBackwardCall(a, to_dev(h), rstd, wt, b, dx=a if which == "dn" else b,
                                            dweight=acc, accumulate=True)()
        assert torch.equal(dx2, dx)
        assert torch.equal(dw2, 0.5 + dw)


@pytest.mark.parametrize("m,k", [(1, 4), (3, 16), (5, 132), (70, 2048), (2, 14332)])
def test_restore_activations(bl, m, k):
    rng = np.random.default_rng([6, m, k])
    q = rng.integers(-128, 128, (m, k)).astype(np.int8)
    s = (127 / np.exp(3 * rng.standard_normal(m))).astype(np.float32)
    s[0] = np.float32(127) / np.float32(1e-5)
    got = bl.restore_activations(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV))
    assert np.array_equal(bits_of(got), ref.restore_activations(q, s))


# ------------------------------------------------------------------ gradients of BitLinear

def layer_case(bl, seed, m, n, k):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16)
    q, xs = bl.act_quant(x)
    packed, ws = bl.pack_weights(0.02 * torch.randn(n, k, generator=g, device=DEV))
    dy = torch.randn(m, n, generator=g, device=DEV) * torch.exp(torch.randn(m, 1, generator=g, device=DEV))
    dy[2::5] = 0  # tokens that the loss masks out
    return dy.to(torch.bfloat16), q, xs, packed, ws


def input_gradient(bl, dy, packed, ws):
    u = bl.unpack_weights(packed).double()
    return dy.double() @ u / ws.double(), dy.double().abs() @ u.abs() / ws.double()


def weight_gradient(bl, dy, q, xs):
    xhat = bl.restore_activations(q, xs).double()
    d = dy.double().t().contiguous()
    return d @ xhat, d.abs() @ xhat.abs()


def check_input(got, want, mag, n):
    tol = BF * want.abs() + (1 + BF) * (n + 2) * 2 * U * mag
    assert bool(((got.double() - want).abs() <= tol).all())


def check_weight(got, want, mag, m):
    assert bool(((got.double() - want).abs() <= (m + 2) * 2 * U * mag).all())


BACKWARD_SHAPES = [(1, 1, 4), (1, 16, 64), (3, 5, 12), (64, 64, 64), (65, 130, 68), (17, 8, 2052),
                   (130, 257, 516), (301, 1001, 1284), (2, 4096, 4096), (40, 2048, 2048),
                   (700, 24, 24), (4096, 72, 4096), (72, 4096, 4100)]


@pytest.mark.parametrize("m,n,k", BACKWARD_SHAPES)
def test_backward(bl, m, n, k):
    dy, q, xs, packed, ws = layer_case(bl, 10 + m, m, n, k)
    call = bl.BackwardCall(dy, q, xs, packed, ws, bias=True)
    dx, dw, db = call()
    check_input(dx, *input_gradient(bl, dy, packed, ws), n)
    check_weight(dw, *weight_gradient(bl, dy, q, xs), m)
    d = dy.double()
    assert bool(((db.double() - d.sum(0)).abs() <= (m + 2) * U * d.abs().sum(0)).all())
    first = [t.clone() for t in (dx, dw, db)]
    for a, b in zip(call(), first):  # the same bits every time
        assert torch.equal(a, b)


@pytest.mark.parametrize("m,n,k", [(5, 16, 256), (40, 48, 512), (130, 272, 2048), (1, 4096, 1024)])
def test_backward_input_tiled_layout(bl, m, n, k):
    dy, q, xs, packed, ws = layer_case(bl, 20 + m, m, n, k)
    assert torch.equal(bl.backward_input(dy, bl.tile_weights(packed), ws, k=k),
                       bl.backward_input(dy, packed, ws))


def test_backward_shared_input_adds_up(bl):
    """Layers that share an input: each adds to the gradient in place, rounded
    to bf16 as a bf16 tensor add."""
    dy, q, xs, packed, ws = layer_case(bl, 31, 33, 72, 260)
    dx = bl.backward_input(dy, packed, ws)
    prev = torch.randn(33, 260, device=DEV).to(torch.bfloat16)
    want = dx + prev
    out = prev.clone()
    bl.backward_input(dy, packed, ws, residual=out, out=out)
    assert torch.equal(out, want)
    assert torch.equal(bl.backward_input(dy, packed, ws, residual=prev), want)


def test_backward_weight_accumulates(bl):
    dy, q, xs, packed, ws = layer_case(bl, 32, 100, 130, 132)
    dw, db = bl.backward_weight(dy, q, xs, bias=True)
    a, b = torch.full_like(dw, 0.25), torch.full_like(db, -2.0)
    bl.backward_weight(dy, q, xs, out=a, dbias=b, accumulate=True)
    assert torch.equal(a, dw + 0.25) and torch.equal(b, db - 2.0)


def test_backward_not_finite_stays_in_its_row(bl):
    """An infinity in one token's gradient reaches that token's dx alone."""
    dy, q, xs, packed, ws = layer_case(bl, 33, 70, 136, 68)
    clean = bl.backward_input(dy, packed, ws)
    dy[4, 135] = float("inf")
    got = bl.backward_input(dy, packed, ws)
    keep = torch.arange(70, device=DEV) != 4
    assert torch.equal(got[keep], clean[keep])


# Shapes by the kernels they take: one launch; operand pass and 64 or 128 tiles;
# dx in parts; dw in parts; 128 tiles; 256 tiles with dx in parts.
PLANS = [(33, 72, 260), (512, 1024, 1024), (45, 4000, 480), (2048, 512, 512), (300, 4096, 4096), (2048, 6912, 2560)]


@pytest.mark.parametrize("m,n,k", PLANS)
def test_backward_options_on_every_plan(bl, m, n, k):
    """Residual in place, accumulation, the tiled layout and a value that is not
    finite, against the plain call of the same shape."""
    dy, q, xs, packed, ws = layer_case(bl, 60 + m, m, n, k)
    dx, dw, db = bl.BackwardCall(dy, q, xs, packed, ws, bias=True)()
    check_input(dx, *input_gradient(bl, dy, packed, ws), n)
    check_weight(dw, *weight_gradient(bl, dy, q, xs), m)
    prev = torch.randn(m, k, device=DEV).to(torch.bfloat16)
    rx, rw, rb = prev.clone(), torch.full_like(dw, 0.5), torch.full_like(db, -1.0)
    bl.BackwardCall(dy, q, xs, packed, ws, residual=rx, dx=rx, dw=rw, dbias=rb, accumulate=True)()
    assert torch.equal(rx, dx + prev) and torch.equal(rw, dw + 0.5) and torch.equal(rb, db - 1.0)
    if n % 16 == 0 and k % 256 == 0:
        tx, tw, _ = bl.BackwardCall(dy, q, xs, bl.tile_weights(packed), ws)()
        assert torch.equal(tx, dx) and torch.equal(tw, dw)
    bad = dy.clone()
    bad[m // 2, n - 1] = float("nan")
    bx, bw, _ = bl.BackwardCall(bad, q, xs, packed, ws)()
    rows, cols = torch.arange(m, device=DEV) != m // 2, torch.arange(n, device=DEV) != n - 1
    assert torch.equal(bx[rows], dx[rows]) and torch.equal(bw[cols], dw[cols])


@pytest.mark.parametrize("m,n,k", PLANS)
def test_backward_leaves_what_is_behind(bl, m, n, k):
    """Rows behind the outputs' last stay as they were."""
    dy, q, xs, packed, ws = layer_case(bl, 70 + m, m, n, k)
    dx = torch.full((m + 2, k), 7.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((n + 2, k), 7.0, device=DEV)
    db = torch.full((n + 8,), 7.0, device=DEV)
    bl.BackwardCall(dy, q, xs, packed, ws, dx=dx[:m], dw=dw[:n], dbias=db[:n])()
    assert bool((dx[m:] == 7).all()) and bool((dw[n:] == 7).all()) and bool((db[n:] == 7).all())


# ------------------------------------------------------------------ 4-bit weights

@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (16, 128, 128), (17, 160, 32), (5, 192, 64),
                                       (33, 256, 256), (20, 1024, 1024), (48, 2048, 512)])
def test_w4_pack(bl, n, k, group):
    rng = np.random.default_rng([7, n, k])
    w = (rng.standard_normal((n, k)) * 0.02).astype(np.float32)
    w[0, :group] = 0  # a group of zeros
    w[-1, -group:] *= 1e-3
    p = bl.pack_weights_w4(torch.from_numpy(w).to(DEV), group)
    v, s = ref.w4_quant(w, group)
    codes, scales = ref.w4_pack(v, s)
    assert np.array_equal(p.codes.cpu().numpy().reshape(-1), codes)
    assert np.array_equal(bits_of(p.scales).reshape(-1), scales)
    full = v.astype(np.float32) * np.repeat(oracle.bf16_to_f32(s), group, axis=1)
    assert np.array_equal(bl.unpack_weights_w4(p).cpu().numpy(), full)
    # half a step of the group's scale, and the scale's own rounding at the
    # largest value (7 s against max|w|: 2^-8 of it)
    amax = np.repeat(np.abs(w.reshape(n, -1, group)).max(2), group, axis=1)
    assert np.all(np.abs(full - w) <= amax / 14 * (1 + 2 * BF) + amax * BF)


def w4_case(bl, seed, m, n, k, group):
    rng = np.random.default_rng([8, seed])
    q = rng.integers(-127, 128, (m, k)).astype(np.int8)
    q[2::3] = 0
    xs = (127 / np.exp(rng.standard_normal(m))).astype(np.float32)
    w = torch.from_numpy((rng.standard_normal((n, k)) * 0.02).astype(np.float32)).to(DEV)
    return torch.from_numpy(q).to(DEV), torch.from_numpy(xs).to(DEV), bl.pack_weights_w4(w, group)


def w4_reference(bl, q, xs, p):
    """y before rounding, and the sum of the group terms' magnitudes."""
    m, g = q.shape[0], p.k // p.group
    w = bl.unpack_weights_w4(p).double()
    y, mag = torch.zeros(m, p.n, dtype=torch.float64, device=DEV), torch.zeros(m, p.n, dtype=torch.float64, device=DEV)
    step = min(p.group, 128)  # a group over 128 is added up 128 at a time
    for i in range(p.k // step):
        t = q[:, i * step:(i + 1) * step].double() @ w[:, i * step:(i + 1) * step].t().contiguous()
        y += t
        mag += t.abs()
    return y / xs.double()[:, None], mag / xs.double()[:, None]


@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("m,n,k", [(1, 1, 256), (1, 16, 1024), (3, 35, 768), (16, 1003, 2304), (17, 64, 512),
                                   (1, 4096, 4096), (5, 2048, 14336), (40, 128, 4352), (2, 8192, 256)])
def test_w4_forward(bl, m, n, k, group):
    q, xs, p = w4_case(bl, m + n, m, n, k, group)
    bias = torch.randn(n, device=DEV).to(torch.bfloat16)
    y = bl.forward_w4(q, xs, p)
    want, mag = w4_reference(bl, q, xs, p)
    # exact integers within a group; one fp32 product and sum per group, a
    # division, the rounding to bf16
    tol = BF * want.abs() + (1 + BF) * (2 * (k // min(group, 128)) + 8) * U * mag
    assert bool(((y.double() - want).abs() <= tol).all())
    assert torch.equal(bl.forward_w4(q, xs, p, bias=bias), y + bias)


@pytest.mark.parametrize("k,group", [(32, 32), (96, 32), (64, 64), (2080, 32), (192, 64), (8256, 64)])
def test_w4_forward_short_tiles(bl, k, group):
    """K that ends inside a tile of 128."""
    q, xs, p = w4_case(bl, k, 7, 50, k, group)
    y = bl.forward_w4(q, xs, p)
    want, mag = w4_reference(bl, q, xs, p)
    tol = BF * want.abs() + (1 + BF) * (2 * (k // group) + 8) * U * mag
    assert bool(((y.double() - want).abs() <= tol).all())


def test_w4_forward_leaves_other_rows(bl):
    q, xs, p = w4_case(bl, 3, 5, 37, 256, 64)
    y = torch.full((9, 37), 7.0, dtype=torch.bfloat16, device=DEV)
    bl.forward_w4(q, xs, p, out=y[:5])
    assert bool((y[5:] == 7).all())


# ------------------------------------------------------------------ streams and graphs

def test_operators_on_a_side_stream_and_in_a_graph(bl):
    """Norm, 4-bit product and the gradients, captured together and replayed on
    new inputs: every replay against the eager result."""
    m, n, k = 24, 96, 512
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16)
    r = torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16)
    w = (1 + 0.1 * torch.randn(k, generator=g, device=DEV))
    w4 = bl.pack_weights_w4(torch.randn(n, k, generator=g, device=DEV), 64)
    packed, ws = bl.pack_weights(torch.randn(n, k, generator=g, device=DEV))
    norm = bl.NormQuantCall(x, w, r)
    head = bl.W4Call(norm.out.q, norm.out.x_scale, w4)
    back = bl.BackwardCall(head.out, norm.out.q, norm.out.x_scale, packed, ws, bias=True)
    dx, dw, db = back()
    nback = bl.NormQuantBackwardCall(dx, norm.out.h, norm.out.rstd, w)

    def step():
        norm()
        head()
        back()
        nback()
        return [norm.out.q, norm.out.x_scale, norm.out.h, head.out, dx, dw, db,
                nback.dx, nback.dweight]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(torch.randn(m, k, generator=g, device=DEV))
        want = [t.clone() for t in step()]
        for t in step():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [norm.out.q, norm.out.x_scale, norm.out.h, head.out, dx, dw, db,
               nback.dx, nback.dweight]
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


def test_a_side_stream_waits_for_nothing_else(bl):
    """Calls go to the current stream: results on a side stream, read there."""
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(64, 1024, generator=g, device=DEV).to(torch.bfloat16)
    want = bl.rms_norm_quant(x)
    dy, q, xs, packed, ws = layer_case(bl, 40, 64, 512, 1024)
    first = bl.BackwardCall(dy, q, xs, packed, ws)()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = bl.rms_norm_quant(x)
        again = bl.BackwardCall(dy, q, xs, packed, ws)()
        same = [torch.equal(a, b) for a, b in zip(got[:4], want[:4])]
        same += [torch.equal(a, b) for a, b in zip(again[:2], first[:2])]
    side.synchronize()
    assert all(same)


def test_concurrent_calls_from_threads(bl):
    """Several host threads, each on its own stream and workspaces."""
    import threading

    cases = [layer_case(bl, 50 + i, 40 + 100 * i, 256, 1024) for i in range(4)]
    want = [[t.clone() for t in bl.BackwardCall(*c, bias=True)()] for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                call = bl.BackwardCall(*cases[i], bias=True)
                for _ in range(10):
                    got = call()
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


# ------------------------------------------------------------------ offsets past 2^31 and 2^32

def test_norm_far_rows(bl):
    """Rows past 2^31 elements (2^32 bytes) are those of a call on them alone."""
    k = 4100
    m = 2 ** 31 // k + 5
    x = torch.empty(m, k, dtype=torch.bfloat16, device=DEV)
    x[:-8] = 1.0
    x[-8:] = torch.randn(8, k, device=DEV).to(torch.bfloat16)
    w = torch.randn(k, device=DEV)
    got = bl.rms_norm_quant(x, w)
    few = bl.rms_norm_quant(x[-8:].clone(), w)
    for a, b in zip((got.q, got.x_scale, got.rstd), (few.q, few.x_scale, few.rstd)):
        assert torch.equal(a[-8:], b)
    xhat = bl.restore_activations(got.q, got.x_scale)
    assert torch.equal(xhat[-8:], bl.restore_activations(few.q, few.x_scale))
    del xhat
    dn = torch.zeros_like(x)
    dn[-8:] = torch.randn(8, k, device=DEV).to(torch.bfloat16)
    dx, dw = bl.rms_norm_quant_backward(dn, x, got.rstd, w)
    dx2, dw2 = bl.rms_norm_quant_backward(dn[-8:].clone(), x[-8:].clone(), few.rstd, w)
    assert torch.equal(dx[-8:], dx2)
    assert bool(((dw - dw2).abs() <= 16 * U * (dn[-8:].double() * x[-8:].double() * few.rstd.double()[:, None]).abs().sum(0)).all())


def test_backward_far_weights(bl):
    """Weights past 2^31 elements: the last rows' gradient, and an input
    gradient that sums over all of them."""
    m, k = 3, 36864
    n = 2 ** 31 // k + 64
    n += -n % 16
    g = torch.Generator(device=DEV).manual_seed(3)
    packed = torch.full((n, k // 4), 0x55, dtype=torch.uint8, device=DEV)  # zeros
    w = 0.02 * torch.randn(32, k, generator=g, device=DEV)
    tail, ws = bl.pack_weights(w)
    packed[-32:] = tail
    dy = torch.randn(m, n, generator=g, device=DEV).to(torch.bfloat16)
    q, xs = bl.act_quant(torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16))
    dx, dw, _ = bl.BackwardCall(dy, q, xs, packed, ws)()
    last = dy[:, -32:].contiguous()
    check_input(dx, *input_gradient(bl, last, tail, ws), n)
    check_weight(dw[-32:], *weight_gradient(bl, last, q, xs), m)
    check_weight(dw[:32], *weight_gradient(bl, dy[:, :32].contiguous(), q, xs), m)


def test_w4_far_weights(bl):
    """4-bit codes past 2^31 bytes: the last rows' outputs."""
    k, group = 8192, 128
    n = 2 ** 31 // (k // 2) + 48
    g = torch.Generator(device=DEV).manual_seed(4)
    tail = bl.pack_weights_w4(torch.randn(32, k, generator=g, device=DEV), group)
    codes = torch.zeros(n // 16, k // 128, 4, 16, 16, dtype=torch.uint8, device=DEV)
    scales = torch.ones(n // 16, k // group, 16, dtype=torch.bfloat16, device=DEV)
    codes[-2:], scales[-2:] = tail.codes, tail.scales
    q = torch.randint(-127, 128, (2, k), generator=g, device=DEV).to(torch.int8)
    xs = torch.ones(2, device=DEV)
    y = bl.forward_w4(q, xs, bl.W4Weights(codes, scales, n, k, group))
    want, mag = w4_reference(bl, q, xs, tail)
    assert bool(((y[:, -32:].double() - want).abs() <= BF * want.abs() + (1 + BF) * (2 * (k // group) + 8) * U * mag).all())
    assert bool((y[:, :-32] == 0).all())


# ------------------------------------------------------------------ every kernel and plan of the gradients

# Per shape the plan that its gradients take, of both together, of dx alone and of
# dw alone: "one" for the one-launch kernel, else the tiles of dx and dw and the
# parts of their sums (None: not wanted).  test_layer_host.py holds the plan to
# this, so that other costs in it cannot leave a kernel without a test.
BY_PLAN = {
    # 256 tiles, ragged in M, N and K; dy laid out; dw stored past the caches
    (1500, 2050, 4100): ((256, 1, 256, 1), (128, 1, None, None), (None, None, 128, 1)),
    # the same with dx past the caches too, and a last slab of one token
    (2049, 1500, 14332): ((256, 1, 256, 1), (256, 1, None, None), (None, None, 128, 1)),
    # 256 tiles in parts: dx, dw, either alone, whole sizes
    (2050, 6900, 2564): ((256, 2, 256, 1), (128, 2, None, None), (None, None, 128, 1)),
    (8190, 2050, 2500): ((256, 1, 256, 2), (128, 1, None, None), (None, None, 128, 3)),
    (1800, 8100, 2308): ((128, 1, 128, 1), (256, 3, None, None), (None, None, 128, 1)),
    (8300, 1900, 1924): ((128, 1, 128, 1), (128, 1, None, None), (None, None, 256, 4)),
    (8192, 2048, 2048): ((256, 1, 256, 2), (256, 1, None, None), (None, None, 256, 4)),
    # 128 tiles, whole sums and in parts
    (1025, 2050, 4100): ((128, 1, 128, 1), (128, 1, None, None), (None, None, 128, 1)),
    (4100, 700, 2052): ((128, 1, 128, 2), (128, 1, None, None), (None, None, 128, 2)),
    (200, 5000, 1028): ((128, 8, 128, 1), (64, 6, None, None), (None, None, 128, 1)),
    # 64 and 128 tiles in one launch
    (700, 5000, 1284): ((64, 1, 128, 1), (64, 2, None, None), (None, None, 128, 1)),
    (1100, 1100, 1100): ((128, 1, 64, 1), "one", (None, None, 64, 1)),
    # 64 tiles
    (600, 600, 600): ((64, 1, 64, 1), "one", (None, None, 64, 1)),
    (129, 3001, 516): ((64, 6, 64, 1), (64, 8, None, None), "one"),
    (3001, 129, 516): ((64, 1, 64, 6), "one", (None, None, 64, 8)),
    # rows of weights shorter than a dword of the two-bit transpose's
    (1, 2097152, 4): ((64, 16, 128, 1), (64, 16, None, None), (None, None, 128, 1)),
    (4000, 4097, 8): ((64, 4, 64, 4), (64, 8, None, None), (None, None, 64, 6)),
    (4000, 4097, 12): ((64, 4, 64, 4), (64, 8, None, None), (None, None, 64, 6)),
}


@pytest.mark.parametrize("m,n,k", list(BY_PLAN))
def test_backward_by_plan(bl, m, n, k):
    """Options, rows behind the outputs, and each gradient by itself."""
    test_backward_options_on_every_plan(bl, m, n, k)
    test_backward_leaves_what_is_behind(bl, m, n, k)
    dy, q, xs, packed, ws = layer_case(bl, 80 + m, m, n, k)
    check_input(bl.backward_input(dy, packed, ws), *input_gradient(bl, dy, packed, ws), n)
    dw, db = bl.backward_weight(dy, q, xs, bias=True)
    check_weight(dw, *weight_gradient(bl, dy, q, xs), m)
    d = dy.double()
    assert bool(((db.double() - d.sum(0)).abs() <= (m + 2) * U * d.abs().sum(0)).all())


# Shapes whose gradients go through a workspace: 64 tiles, sums of dx in parts, of
# dw in parts, 64 and 128 tiles.
STAGED = [(600, 600, 600), (45, 4000, 480), (2048, 512, 512), (300, 1000, 2052)]


def workspace_bytes(bl, m, n, k):
    return bl.lib().bitlinear_backward_workspace_bytes(m, n, k, 1, 1)


@pytest.mark.parametrize("m,n,k", STAGED)
def test_staged_gradients_in_a_graph(bl, m, n, k):
    """Operand pass, products and the sum of the parts, and the norm's gradient
    with its second launch, captured with the forward calls around them and
    replayed on new inputs: every replay against the eager result."""
    assert workspace_bytes(bl, m, n, k) > 0
    assert bl.lib().bitlinear_rms_norm_quant_backward_workspace_bytes(m, k, 1) > 0
    g = torch.Generator(device=DEV).manual_seed(m)
    x, r = (torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    dy = torch.randn(m, n, generator=g, device=DEV).to(torch.bfloat16)
    w = 1 + 0.1 * torch.randn(k, generator=g, device=DEV)
    packed, ws = bl.pack_weights(torch.randn(n, k, generator=g, device=DEV))
    norm = bl.NormQuantCall(x, w, r)
    product = bl.GroupedQuantizedCall([norm.out.q], [norm.out.x_scale], [packed], [ws])
    back = bl.BackwardCall(dy, norm.out.q, norm.out.x_scale, packed, ws, bias=True)
    nback = bl.NormQuantBackwardCall(back._out[0], norm.out.h, norm.out.rstd, w)
    outs = [norm.out.q, norm.out.x_scale, norm.out.h, product.outs[0], *back._out, nback.dx, nback.dweight]

    def step():
        norm()
        product()
        back()
        nback()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(torch.randn(m, k, generator=g, device=DEV))
        dy.copy_(torch.randn(m, n, generator=g, device=DEV))
        step()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), i


def test_graphs_that_share_a_workspace(bl):
    """Gradients of several shapes captured over one workspace and replayed one
    after the other, in changing order: each leaves nothing to the next."""
    cases = [layer_case(bl, 90 + i, *s) for i, s in enumerate(STAGED)]
    workspace = torch.empty(max(workspace_bytes(bl, *s) for s in STAGED), dtype=torch.uint8, device=DEV)
    calls = [bl.BackwardCall(*c, bias=True, workspace=workspace) for c in cases]
    want = [[t.clone() for t in call()] for call in calls]
    graphs = []
    for call in calls:
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for order in ([0, 1, 2, 3], [3, 1, 0, 2], [2, 2, 3, 0]):
        for i in order:
            for t in calls[i]._out:
                t.zero_()
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in order:
            assert all(torch.equal(a, b) for a, b in zip(calls[i]._out, want[i])), (order, i)


def test_staged_gradients_on_side_streams(bl):
    """Calls with workspaces of their own, in turn on four streams that run at
    the same time."""
    cases = [layer_case(bl, 95 + i, *s) for i, s in enumerate(STAGED)]
    assert all(workspace_bytes(bl, *s) > 0 for s in STAGED)
    want = [[t.clone() for t in bl.BackwardCall(*c, bias=True)()] for c in cases]
    torch.cuda.synchronize()
    streams, calls, got = [torch.cuda.Stream() for _ in cases], [], [[] for _ in cases]
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            calls.append(bl.BackwardCall(*c, bias=True))
    assert len({c.workspace.data_ptr() for c in calls}) == len(calls)
    for _ in range(20):
        for i, (call, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i].append([t.clone() for t in call()])
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        assert all(torch.equal(a, b) for out in outs for a, b in zip(out, want[i])), STAGED[i]


def test_staged_gradients_from_threads(bl):
    """Host threads, each with a shape, stream and workspace of its own, every
    call's results kept and checked."""
    import threading

    assert all(workspace_bytes(bl, *s) > 0 for s in STAGED)
    cases = [layer_case(bl, 100 + i, *s) for i, s in enumerate(STAGED)]
    want = [[t.clone() for t in bl.BackwardCall(*c, bias=True)()] for c in cases]
    torch.cuda.synchronize()
    bad, together = [], threading.Barrier(len(cases))

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                call = bl.BackwardCall(*cases[i], bias=True)
                together.wait(timeout=30)
                got = [[t.clone() for t in call()] for _ in range(20)]
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for out in got for a, b in zip(out, want[i])):
                    bad.append(STAGED[i])
        except Exception as e:  # reported by the main thread
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


# ------------------------------------------------------------------ the other kernels and rules

# Rows over 32768 columns are read three times; over 256 tokens a thread takes two
# pieces from 4096 columns on, and four from 8192.
LONG_ROWS = [(3, 32772), (2, 65536), (5, 100004), (1, 2 ** 20 + 4), (300, 4104), (300, 8192), (260, 14332)]


@pytest.mark.parametrize("weight", ["none", "bf16", "fp32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("m,k", LONG_ROWS)
def test_norm_quant_long_rows(bl, m, k, residual, weight):
    test_norm_quant(bl, m, k, residual, weight)


@pytest.mark.parametrize("k", [32772, 70000])
def test_norm_long_rows_in_place_and_not_finite(bl, k):
    for which in ("x", "residual"):
        test_norm_quant_in_place(bl, k, which)
    test_norm_not_finite_stays_in_its_row(bl, k)
    # without h, the sum with the residual is made again for each reading
    rng = np.random.default_rng([7, k])
    x, r = to_dev(rows(rng, 3, k)), to_dev(rows(rng, 3, k, 3.0))
    want = bl.rms_norm_quant(x, None, r, want_norm=True)
    n, rstd = torch.empty_like(x), torch.empty(4, device=DEV)
    bl._launch(bl.lib().bitlinear_rms_norm_quant,
               (3, k, x.data_ptr(), r.data_ptr(), None, 0, 1e-6, None, rstd.data_ptr(), n.data_ptr(), None, None),
               x.device)
    assert torch.equal(n, want.n) and torch.equal(rstd[:3], want.rstd)


def test_norm_many_rows(bl):
    """Rows past 2^20: the grid's second dimension."""
    m, k = 2 ** 20 + 5, 64
    x = torch.randn(m, k, device=DEV).to(torch.bfloat16)
    got = bl.rms_norm_quant(x, want_norm=True)
    for part in (slice(0, 9), slice(2 ** 20 - 4, m)):
        few = bl.rms_norm_quant(x[part].contiguous(), want_norm=True)
        for a, b in zip((got.q, got.x_scale, got.rstd, got.n), (few.q, few.x_scale, few.rstd, few.n)):
            assert torch.equal(a[part], b)
    assert bool((got.x_scale > 0).all())
    xhat = bl.restore_activations(got.q, got.x_scale)
    assert torch.equal(xhat[-9:], bl.restore_activations(got.q[-9:].contiguous(), got.x_scale[-9:].clone()))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", [(5, 16392, 256), (16, 16400, 4352), (7, 32776, 512), (21, 32800, 384), (16, 65544, 256)])
def test_w4_forward_many_rows(bl, m, n, k, group):
    """Blocks of 16 rows by four, two and one waves (more than four tokens
    through 16384 rows and more), the last ones partly filled."""
    test_w4_forward(bl, m, n, k, group)


def test_w4_far_outputs(bl):
    """Outputs past 2^31: the last tokens'."""
    m, n, k, group = 2 ** 18 + 7, 8200, 64, 32
    q, xs, p = w4_case(bl, 9, 23, n, k, group)
    big = torch.zeros(m, k, dtype=torch.int8, device=DEV)
    big[-23:] = q
    scales = torch.ones(m, device=DEV)
    scales[-23:] = xs
    y = bl.forward_w4(big, scales, p)
    assert torch.equal(y[-23:], bl.forward_w4(q, xs, p))
    assert not bool(y[:-23].any())


def test_backward_far_tokens(bl):
    """Inputs past 2^31 elements: the last tokens' gradient, and a weight
    gradient that sums over all of them."""
    m, n, k, last = 2 ** 19 + 67, 72, 4100, 33
    dy, q, xs, packed, ws = layer_case(bl, 110, last, n, k)
    big_dy = torch.zeros(m, n, dtype=torch.bfloat16, device=DEV)
    big_q = torch.ones(m, k, dtype=torch.int8, device=DEV)
    big_xs = torch.ones(m, device=DEV)
    big_dy[-last:], big_q[-last:], big_xs[-last:] = dy, q, xs
    res = torch.zeros(m, k, dtype=torch.bfloat16, device=DEV)
    res[-last:] = 2.0
    dx, dw, db = bl.BackwardCall(big_dy, big_q, big_xs, packed, ws, bias=True, residual=res, dx=res)()
    alone = bl.BackwardCall(dy, q, xs, packed, ws, bias=True)()
    # rounded twice against once: both sums hold the bound before that
    want, mag = input_gradient(bl, dy, packed, ws)
    tol = 2 * BF * (want.abs() + 2) + (1 + 2 * BF) * (n + 2) * 2 * U * mag
    assert bool(((dx[-last:].double() - (want + 2)).abs() <= tol).all())
    assert not bool(dx[:-last].any())
    check_input(alone[0], want, mag, n)
    check_weight(dw, *weight_gradient(bl, dy, q, xs), last)
    assert bool(((db.double() - dy.double().sum(0)).abs() <= (last + 2) * U * dy.double().abs().sum(0)).all())


@pytest.mark.parametrize("m", [1, 9])
@pytest.mark.parametrize("k,group", [(64, 32), (256, 64), (512, 128), (2048, 1024)])
def test_w4_weights_that_are_not_finite(bl, m, k, group):
    """A weight that is not a number, or infinite, spoils its group's scale and all of
    that output's values, and no others."""
    torch.manual_seed(76)
    n = 37
    x = torch.randn(m, k, device=DEV).to(torch.bfloat16)
    q, xs = bl.act_quant(x)
    w = 0.02 * torch.randn(n, k, device=DEV)
    good = bl.pack_weights_w4(w, group)
    y, u = bl.forward_w4(q, xs, good), bl.unpack_weights_w4(good)
    for value in (float("nan"), float("inf"), -float("inf")):
        for at in (0, group - 1, k - 1):
            bad = w.clone()
            bad[20, at] = value
            p = bl.pack_weights_w4(bad, group)
            others = [i for i in range(n) if i != 20]
            scales = bl.unpack_weights_w4(p)
            g = at // group * group
            assert not bool(torch.isfinite(scales[20, g:g + group]).any())
            rest = [i for i in range(k) if not g <= i < g + group]
            assert torch.equal(scales[20, rest], u[20, rest]) and torch.equal(scales[others], u[others])
            got = bl.forward_w4(q, xs, p)
            assert not bool(torch.isfinite(got[:, 20]).any()) and torch.equal(got[:, others], y[:, others])
