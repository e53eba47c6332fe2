"""The training form (training.py) on the GPU: values against the inference
path, gradients against the formulas in float64 and against differences of the
straight-through function, and the operators run together as a block uses them.

Bounds count roundings: u = 2^-24 a half step of fp32 (a whole one, 2u, per term
of a matrix-core sum), 2^-8 one of bf16, relative.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
U, BF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def bl():
    from bit_gemm_bitlinear_amd import bitlinear

    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return bitlinear


@pytest.fixture(scope="module")
def tr(bl):
    from bit_gemm_bitlinear_amd import training

    return training


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def leaf(shape, g, dtype=torch.bfloat16, scale=1.0):
    return (scale * torch.randn(shape, generator=g, device=DEV)).to(dtype).requires_grad_()


@pytest.mark.parametrize("shape,n,bias", [((1, 64), 16, False), ((5, 7, 132), 33, True), ((40, 1024), 96, True)])
def test_linear(bl, tr, shape, n, bias):
    g = gen(1)
    k = shape[-1]
    x, w = leaf(shape, g), leaf((n, k), g, torch.float32, 0.02)
    b = leaf((n,), g) if bias else None
    y = tr.linear(x, w, b)
    rows = x.detach().reshape(-1, k)
    packed, ws = bl.pack_weights(w.detach())
    assert torch.equal(y.detach().reshape(-1, n), bl.forward(rows, packed, ws, bias=None if b is None else b.detach()))
    dy = torch.randn(y.shape, generator=g, device=DEV).to(torch.bfloat16)
    y.backward(dy)
    d = dy.reshape(-1, n).double()
    q, xs = bl.act_quant(rows)
    u, xhat = bl.unpack_weights(packed).double(), bl.restore_activations(q, xs).double()
    want = d @ u / ws.double()
    mag = d.abs() @ u.abs() / ws.double()
    assert x.grad.shape == x.shape
    assert bool(((x.grad.reshape(-1, k).double() - want).abs() <= BF * want.abs() + (1 + BF) * (n + 2) * 2 * U * mag).all())
    dt = d.t().contiguous()
    assert bool(((w.grad.double() - dt @ xhat).abs() <= (len(rows) + 2) * 2 * U * (dt.abs() @ xhat.abs())).all())
    if bias:
        s = d.sum(0)
        assert bool(((b.grad.double() - s).abs() <= BF * s.abs() + (1 + BF) * (len(rows) + 2) * U * d.abs().sum(0)).all())


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("weight", ["none", "bf16", "fp32"])
def test_norm_linear(bl, tr, weight, residual):
    """Three projections of one norm's output; the middle one's output unused."""
    g = gen(2)
    m, k, ns = 50, 516, (64, 8, 130)
    x = leaf((2, 25, k), g)
    r = leaf((2, 25, k), g, scale=2.0) if residual else None
    nw = None if weight == "none" else leaf((k,), g, torch.bfloat16 if weight == "bf16" else torch.float32)
    ws = [leaf((n, k), g, torch.float32, 0.02) for n in ns]
    b = leaf((ns[2],), g)
    h, ys = tr.norm_linear(x, ws, nw, r, biases=[None, None, b], eps=1e-5)
    x2 = x.detach().reshape(m, k)
    normed = bl.rms_norm_quant(x2, None if nw is None else nw.detach(), None if r is None else r.detach().reshape(m, k),
                               eps=1e-5, want_norm=True)
    packs = [bl.pack_weights(w.detach()) for w in ws]
    assert torch.equal(h.detach().reshape(m, k), normed.h)
    for i in range(3):  # the codes' product is the product of the norm's bf16 output
        want = bl.forward(normed.n, *packs[i], bias=b.detach() if i == 2 else None)
        assert torch.equal(ys[i].detach().reshape(m, ns[i]), want)
    dys = [torch.randn(y.shape, generator=g, device=DEV).to(torch.bfloat16) for y in ys]
    dh = torch.randn(h.shape, generator=g, device=DEV).to(torch.bfloat16)
    torch.autograd.backward([h, ys[0], ys[2]], [dh, dys[0], dys[2]])
    assert ws[1].grad is None
    dx0 = bl.backward_input(dys[0].reshape(m, -1), *packs[0])
    dn = bl.backward_input(dys[2].reshape(m, -1), *packs[2], residual=dx0)
    dx, dweight = bl.rms_norm_quant_backward(dn, normed.h, normed.rstd, None if nw is None else nw.detach(),
                                             dh.reshape(m, k) if residual else None)
    if not residual:  # h is x itself
        dx = dx + dh.reshape(m, k)
    assert torch.equal(x.grad.reshape(m, k), dx)
    if residual:
        assert torch.equal(r.grad.reshape(m, k), dx)
    if nw is not None:
        assert torch.equal(nw.grad, dweight.to(nw.dtype))
    for i in (0, 2):
        dw, db = bl.backward_weight(dys[i].reshape(m, -1), normed.q, normed.x_scale, bias=i == 2)
        assert torch.equal(ws[i].grad, dw)
        if i == 2:
            assert torch.equal(b.grad, db.to(torch.bfloat16))


def test_gradient_against_differences(bl, tr):
    """Directional differences of the straight-through function in float64 (the
    weights' and activations' rounded values held where the forward put them,
    so that it is y = (norm(h) + c) . (w + d)^T with constants c, d)."""
    g = gen(3)
    m, n, k, eps = 12, 40, 256, 1e-5
    x, w, nw = leaf((m, k), g), leaf((n, k), g, torch.float32, 0.02), leaf((k,), g, torch.float32)
    r = leaf((m, k), g)
    h, (y,) = tr.norm_linear(x, [w], nw, r, eps=eps)
    dy = torch.randn(m, n, generator=g, device=DEV).to(torch.bfloat16)
    y.backward(dy)
    normed = bl.rms_norm_quant(x.detach(), nw.detach(), r.detach(), eps=eps)
    xhat = bl.restore_activations(normed.q, normed.x_scale).double()
    packed, ws = bl.pack_weights(w.detach())
    what = bl.unpack_weights(packed).double() / ws.double()

    def value(hh, nn, ww):
        z = hh / torch.sqrt((hh * hh).mean(1, keepdim=True) + eps) * nn
        z = z + (xhat - z0)
        return ((z @ (ww + (what - w.detach().double())).t().contiguous()) * dy.double()).sum()

    h0, n0, w0 = normed.h.double(), nw.detach().double(), w.detach().double()
    z0 = h0 / torch.sqrt((h0 * h0).mean(1, keepdim=True) + eps) * n0
    for got, at in ((x.grad, 0), (nw.grad, 1), (w.grad, 2)):
        d = torch.randn(got.shape, generator=g, device=DEV, dtype=torch.float64)
        t = 1e-5
        args = [[h0, n0, w0], [h0, n0, w0]]
        args[0][at], args[1][at] = args[0][at] + t * d, args[1][at] - t * d
        diff = (value(*args[0]) - value(*args[1])) / (2 * t)
        slope = (got.double() * d).sum()
        # dx passes two roundings to bf16 (of the product's gradient and its
        # own), each off by 2^-8 of a value at most; differences are good to
        # 1e-6 of the terms
        tol = 2 * BF * (got.double().abs() * d.abs()).sum() + 1e-6 * abs(float(diff))
        if at != 2:  # the first rounding, before the norm's gradient takes the mean off
            dn = dy.double() @ what
            back = (dn.abs() * (n0.abs() if at == 0 else 1.0) * normed.rstd.double()[:, None] *
                    (1.0 if at == 0 else h0.abs()))
            tol = tol + 2 * BF * ((back * d.abs()).sum() if at == 0 else (back.sum(0) * d.abs()).sum())
            if at == 0:
                z = h0 * normed.rstd.double()[:, None]
                c = (dn.abs() * n0.abs() * z.abs()).mean(1, keepdim=True)
                tol = tol + 2 * BF * (normed.rstd.double()[:, None] * z.abs() * c * d.abs()).sum()
        assert abs(float(slope - diff)) <= float(tol), at


def test_frozen_inputs(bl, tr):
    g = gen(4)
    x, w = leaf((9, 64), g), leaf((24, 64), g, torch.float32, 0.02)
    tr.linear(x.detach(), w).sum().backward()
    assert w.grad is not None
    wg = w.grad.clone()
    tr.linear(x, w.detach()).sum().backward()
    assert x.grad is not None and torch.equal(w.grad, wg)
    h, (y,) = tr.norm_linear(x.detach(), [w.detach()], None, x.detach())
    assert not h.requires_grad and not y.requires_grad
    r = x.detach().clone().requires_grad_()
    h, _ = tr.norm_linear(x.detach(), [w.detach()], None, r)
    h.sum().backward()  # only the residual stream is used
    assert torch.equal(r.grad, torch.ones_like(r))


def test_second_gradient_is_refused(tr):
    g = gen(5)
    x, w = leaf((4, 64), g), leaf((8, 64), g, torch.float32, 0.02)
    gx, = torch.autograd.grad(tr.linear(x, w).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()


def test_module_and_checkpoint_size(bl, tr):
    """The module's forward is the inference layer's; what it keeps for the
    backward pass is 8 bits an activation and 2 a weight."""
    m, k, n = 256, 1024, 512
    layer = tr.BitLinear(k, n, bias=True, device=DEV)
    x = torch.randn(m, k, device=DEV).to(torch.bfloat16).requires_grad_()
    kept = {}

    def pack(t):
        kept[t.data_ptr()] = t.numel() * t.element_size()
        return t

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        y = layer(x)
    assert sum(kept.values()) <= m * k + 4 * m + n * k // 4 + 4
    frozen = bl.BitLinear(layer.weight.detach(), layer.bias.detach())
    assert torch.equal(frozen(x.detach()), y.detach())
    y.float().square().mean().backward()
    assert layer.weight.grad.shape == layer.weight.shape and layer.bias.grad.dtype == torch.bfloat16


def test_serving_block_together(bl):
    """The decode side together: residual add + norm, the projections on its
    codes, the output head in 4 bits on the same kind of codes."""
    g = gen(6)
    m, d, f, v = 3, 512, 768, 1000
    x = torch.randn(m, d, generator=g, device=DEV).to(torch.bfloat16)
    r = torch.randn(m, d, generator=g, device=DEV).to(torch.bfloat16)
    nw = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16)
    up, us = bl.pack_weights(0.02 * torch.randn(f, d, generator=g, device=DEV))
    down, ds = bl.pack_weights(0.02 * torch.randn(d, f, generator=g, device=DEV))
    head = bl.pack_weights_w4(0.02 * torch.randn(v, d, generator=g, device=DEV), 128)
    a = bl.rms_norm_quant(x, nw, r, want_norm=True)
    up_t = bl.tile_weights(up)
    y = bl.forward_quantized(a.q, a.x_scale, up_t, us)
    assert torch.equal(y, bl.forward(a.n, up, us))
    z = bl.forward(y, down, ds, residual=a.h)
    b = bl.rms_norm_quant(z, nw)
    logits = bl.forward_w4(b.q, b.x_scale, head)
    want = bl.restore_activations(b.q, b.x_scale).double()
    xd = b.q.double() / b.x_scale.double()[:, None]
    w = bl.unpack_weights_w4(head).double().t().contiguous()
    exact = xd @ w
    assert bool(((logits.double() - exact).abs() <= BF * exact.abs() + 20 * U * (xd.abs() @ w.abs())).all())
    # the restored activations are the codes' values to a rounding of bf16
    assert bool(((want - xd).abs() <= BF * xd.abs()).all())


@pytest.mark.parametrize("m", [1, 4, 5, 16, 17, 40, 130, 300])
@pytest.mark.parametrize("n,k", [(64, 256), (33, 260), (17, 516), (1024, 2048)])
def test_forward_quantized_is_the_forward(bl, m, n, k):
    g = gen(m)
    x = torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16)
    if m > 2:
        x[1] = 0
    q, xs = bl.act_quant(x)
    packed, ws = bl.pack_weights(0.02 * torch.randn(n, k, generator=g, device=DEV))
    bias = torch.randn(n, generator=g, device=DEV).to(torch.bfloat16)
    res = torch.randn(m, n, generator=g, device=DEV).to(torch.bfloat16)
    for layout in ([packed, bl.tile_weights(packed)] if n % 16 == 0 and k % 256 == 0 else [packed]):
        assert torch.equal(bl.forward_quantized(q, xs, layout, ws), bl.forward(x, packed, ws))
        assert torch.equal(bl.forward_quantized(q, xs, layout, ws, bias=bias, residual=res),
                           bl.forward(x, packed, ws, bias=bias, residual=res))


def test_grouped_quantized_shares_codes(bl):
    """Projections that share codes, and one on codes of its own, in one call."""
    g = gen(9)
    m = 7
    xa = torch.randn(m, 512, generator=g, device=DEV).to(torch.bfloat16)
    xb = torch.randn(m, 768, generator=g, device=DEV).to(torch.bfloat16)
    ws = [bl.pack_weights(0.02 * torch.randn(n, k, generator=g, device=DEV)) for n, k in ((64, 512), (96, 512), (512, 768))]
    qa, sa = bl.act_quant(xa)
    qb, sb = bl.act_quant(xb)
    got = bl.GroupedQuantizedCall([qa, qa, qb], [sa, sa, sb], [p for p, _ in ws], [s for _, s in ws])()
    want = bl.GroupedCall([xa, xa, xb], [p for p, _ in ws], [s for _, s in ws])()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_training_step_in_a_graph(bl, tr):
    """Forward and backward captured once and replayed on new inputs, each
    replay against the eager step."""
    g = gen(11)
    m, k, n = 96, 512, 160
    x = torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16).requires_grad_()
    r = torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16)
    nw = leaf((k,), g, torch.float32)
    w = [leaf((n, k), g, torch.float32, 0.02) for _ in range(2)]
    target = torch.randn(m, n, generator=g, device=DEV).to(torch.bfloat16)

    def step():
        h, (a, b) = tr.norm_linear(x, w, nw, r)
        return torch.autograd.grad((a, b, h), (x, nw, *w), (target, target, r))

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
            x.copy_(torch.randn(m, k, generator=g, device=DEV))
            target.copy_(torch.randn(m, n, generator=g, device=DEV))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i


def test_same_weight_twice_and_broadcast_input(bl, tr):
    """A weight shared by two projections gets both gradients; a broadcast
    input the sum over its copies."""
    g = gen(12)
    x, w = leaf((1, 256), g), leaf((32, 256), g, torch.float32, 0.02)
    big = x.expand(24, 256)
    h, (a, b) = tr.norm_linear(big, [w, w])
    assert torch.equal(a, b)
    da = torch.randn(24, 32, generator=g, device=DEV).to(torch.bfloat16)
    db = torch.randn(24, 32, generator=g, device=DEV).to(torch.bfloat16)
    torch.autograd.backward([a, b], [da, db])
    normed = bl.rms_norm_quant(big.detach().contiguous())
    each = [bl.backward_weight(d, normed.q, normed.x_scale)[0] for d in (da, db)]
    assert torch.equal(w.grad, each[0] + each[1])
    packed, ws = bl.pack_weights(w.detach())
    dn = bl.backward_input(db, packed, ws, residual=bl.backward_input(da, packed, ws))
    dx, _ = bl.rms_norm_quant_backward(dn, normed.h, normed.rstd)
    s = dx.double().sum(0)
    assert x.grad.shape == x.shape
    # torch adds the 24 rows in bf16 or wider: at most a bf16 rounding a term
    assert bool(((x.grad[0].double() - s).abs() <= 24 * BF * dx.double().abs().sum(0)).all())


def test_slices_off_the_alignment(bl, tr):
    """Inputs and gradients that start off a 16-byte boundary or are strided
    (slices of fused parameters, the parts of a concatenation, a norm weight
    expanded from one value) give what aligned copies of them give."""
    g = gen(8)
    m, k, n = 5, 132, 33

    def parts():
        x = leaf((m + 1, k), g)                  # x[1:] starts 8 bytes past a boundary
        w = leaf((n + 3, k + 4), g, torch.float32, 0.02)
        b = leaf((n + 1,), g)
        nw = leaf((1,), g, torch.float32)
        r = leaf((m, k + 3), g)
        return x, w, b, nw, r

    x, w, b, nw, r = parts()
    views = (x[1:], w[3:, :k], b[1:], nw.expand(k), r[:, 3:])
    copies = [v.detach().clone(memory_format=torch.contiguous_format).requires_grad_() for v in views]
    dys = torch.randn(2 * m + 1, n, generator=g, device=DEV).to(torch.bfloat16)
    dhs = torch.randn(m + 1, k, generator=g, device=DEV).to(torch.bfloat16)

    def run(x, w, b, nw, r, aligned):
        h, (y,) = tr.norm_linear(x, [w], nw, r, biases=[b])
        z = tr.linear(x, w, b)
        # the parts' gradients are slices that start at odd rows of 33 or 132 columns
        if aligned:
            torch.autograd.backward([h, y, z], [dhs[1:].clone(), dys[1:m + 1].clone(), dys[m + 1:].clone()])
        else:
            pad = torch.zeros(1, n, dtype=torch.bfloat16, device=DEV)
            torch.autograd.backward([torch.cat([torch.zeros(1, k, dtype=torch.bfloat16, device=DEV), h]),
                                     torch.cat([pad, y, z])], [dhs, dys])
        return h, y, z

    for a, c in zip(run(*views, aligned=False), run(*copies, aligned=True)):
        assert torch.equal(a, c)
    cx, cw, cb, cn, cr = (c.grad for c in copies)
    assert torch.equal(x.grad[1:], cx) and not bool(x.grad[0].any())
    assert torch.equal(w.grad[3:, :k], cw) and torch.equal(b.grad[1:], cb) and torch.equal(r.grad[:, 3:], cr)
    # 132 sums of one value, by torch: a rounding each
    assert bool((nw.grad.double() - cn.double().sum()).abs() <= 132 * U * cn.double().abs().sum())


# ------------------------------------------------------------------ weights of another width

def test_weight_of_another_width_is_refused(tr):
    """A latent weight must have x's columns; one of sixteen times as many
    has the bytes of a tiled weight with sixteen times the rows."""
    g = gen(13)
    x, r = leaf((4, 256), g), leaf((4, 256), g)
    for shape in ((16, 4096), (16, 1024), (16, 64), (16, 252), (256,), (2, 16, 256)):
        w = leaf(shape, g, torch.float32, 0.02)
        for call in (lambda: tr.linear(x, w), lambda: tr.norm_linear(x, [w]), lambda: tr.norm_linear(x, [w], None, r),
                     lambda: tr.norm_linear(x, [leaf((16, 256), g, torch.float32), w])):
            with pytest.raises(ValueError, match="weight"):
                call()


# ------------------------------------------------------------------ outputs changed in place

@pytest.mark.parametrize("shape", [(6, 64), (2, 3, 64), (64,)])
def test_outputs_change_in_place(tr, shape):
    """Outputs take in-place operations as a torch linear's do, with the
    gradients of the same operations out of place."""
    g = gen(14)
    x, r, b = leaf(shape, g), leaf(shape, g), leaf((24,), g)
    ws = [leaf((24, 64), g, torch.float32, 0.02) for _ in range(2)]
    leaves = (x, r, b, *ws)
    c = torch.randn(*shape[:-1], 24, generator=g, device=DEV).to(torch.bfloat16)

    def grads(in_place):
        add = torch.Tensor.add_ if in_place else torch.Tensor.add
        relu = torch.relu_ if in_place else torch.relu
        y = relu(add(tr.linear(x, ws[0], b), c))
        h, (u, v) = tr.norm_linear(x, ws, None, r)
        u, v = add(u, c), relu(v)
        (z,) = tr.norm_linear(x, [ws[1]])[1]
        z = add(z, c)
        return torch.autograd.grad([(t * t).float().sum() for t in (y, u, v, z, h)], leaves)

    for got, want in zip(grads(True), grads(False)):
        assert torch.equal(got, want)


def test_residual_stream_changed_in_place(tr):
    """h is kept for the backward pass: changed in place it is refused there,
    and an in-place add is the next residual add instead."""
    g = gen(15)
    x, r = leaf((4, 64), g), leaf((4, 64), g)
    w = leaf((24, 64), g, torch.float32, 0.02)
    h, (y,) = tr.norm_linear(x, [w], None, r)
    h.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        (y.float().sum() + h.float().sum()).backward()
    with torch.no_grad():
        h, _ = tr.norm_linear(x, [w], None, r)
        assert torch.equal(h.clone().add_(1), h.add_(1))


@pytest.mark.parametrize("shape", [(6, 64), (2, 3, 64)])
@pytest.mark.parametrize("only_h", [False, True])
def test_gradients_of_x_and_residual_share_no_memory(tr, shape, only_h):
    """Equal gradients, accumulated and changed apart."""
    g = gen(19)
    x, r = leaf(shape, g), leaf(shape, g)
    w = leaf((24, 64), g, torch.float32, 0.02)
    for _ in range(2):
        h, (y,) = tr.norm_linear(x, [w], None, r)
        (h if only_h else y).float().sum().backward()
    once = (torch.ones_like(x) if only_h else
            torch.autograd.grad(tr.norm_linear(x, [w], None, r)[1][0].float().sum(), x)[0])
    assert torch.equal(x.grad, once + once) and torch.equal(r.grad, once + once)
    x.grad.zero_()
    assert torch.equal(r.grad, once + once)


# ------------------------------------------------------------------ no tokens

@pytest.mark.parametrize("shape", [(0, 64), (3, 0, 64)])
def test_no_tokens(tr, shape):
    """A batch without tokens has empty outputs, and every gradient is zero."""
    g = gen(16)
    x, r, b, nw = leaf(shape, g), leaf(shape, g), leaf((24,), g), leaf((64,), g, torch.float32)
    ws = [leaf((24, 64), g, torch.float32, 0.02), leaf((8, 64), g, torch.float32, 0.02)]
    leaves = (x, r, b, nw, *ws)
    y = tr.linear(x, ws[0], b)
    h, (u, v) = tr.norm_linear(x, ws, nw, r, biases=[b, None])
    h2, (z,) = tr.norm_linear(x, [ws[1]], nw)
    assert h2 is x
    for t, n in ((y, 24), (u, 24), (v, 8), (z, 8), (h, 64)):
        assert t.shape == (*shape[:-1], n) and t.dtype == torch.bfloat16 and t.device == x.device
    torch.autograd.backward([y, u, v, z, h], [torch.zeros_like(t) for t in (y, u, v, z, h)])
    for t in leaves:
        assert t.grad.shape == t.shape and t.grad.dtype == t.dtype and not bool(t.grad.any())
    w = leaf((24, 64), g, torch.float32)
    w.grad = torch.ones_like(w)
    tr.BitLinear(64, 24, device=DEV)(x).sum().backward()
    tr.linear(x, w).sum().backward()
    assert bool((w.grad == 1).all())
    with torch.no_grad():
        assert tr.linear(x, w).shape == (*shape[:-1], 24)
    with pytest.raises(ValueError):
        tr.linear(x, leaf((24, 68), g, torch.float32))
    with pytest.raises(TypeError):
        tr.linear(x.float(), w)


# ------------------------------------------------------------------ gradients that are not wanted

def backward_memory(loss):
    """Device memory that the backward pass takes at its largest."""
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    loss.backward()
    torch.cuda.synchronize()
    return torch.cuda.max_memory_allocated() - before


def test_bias_gradient_alone(bl, tr):
    """Over frozen weights the gradient of a bias does not make the weights'."""
    g = gen(17)
    m, n, k = 70, 2048, 4096
    x, w, b = leaf((m, k), g), leaf((n, k), g, torch.float32, 0.02), leaf((n,), g)
    dy = torch.randn(m, n, generator=g, device=DEV).to(torch.bfloat16)
    for inputs in ((x.detach(), w.detach(), b), (x, w.detach(), b)):
        b.grad = x.grad = None
        took = backward_memory((tr.linear(*inputs) * dy).sum())
        s = dy.double().sum(0)
        assert bool(((b.grad.double() - s).abs() <= BF * s.abs() + (1 + BF) * (m + 2) * U * dy.double().abs().sum(0)).all())
        assert took < 4 * n * k
        if inputs[0] is x:
            packed, ws = bl.pack_weights(w.detach())
            assert torch.equal(x.grad, bl.backward_input(dy, packed, ws))


def test_frozen_norm_weight(bl, tr):
    """A frozen norm weight's gradient is not made, nor its workspace."""
    g = gen(18)
    m, n, k = 1100, 16, 8192
    x, w, nw = leaf((m, k), g), leaf((n, k), g, torch.float32, 0.02), leaf((k,), g, torch.float32)
    dy = torch.randn(m, n, generator=g, device=DEV).to(torch.bfloat16)
    took, grads = [], []
    for weight in (nw, nw.detach()):
        x.grad = None
        _, (y,) = tr.norm_linear(x, [w.detach()], weight)
        took.append(backward_memory((y * dy).sum()))
        grads.append(x.grad)
    assert torch.equal(*grads)
    need = bl.lib().bitlinear_rms_norm_quant_backward_workspace_bytes(m, k, 1)
    assert need >= 4 * 512 * k and took[1] <= took[0] - need
    normed = bl.rms_norm_quant(x.detach(), nw.detach())
    dn = torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16)
    dx, dweight = bl.rms_norm_quant_backward(dn, normed.h, normed.rstd, nw.detach(), want_dweight=False)
    assert dweight is None
    assert torch.equal(dx, bl.rms_norm_quant_backward(dn, normed.h, normed.rstd, nw.detach())[0])
    with pytest.raises(ValueError):
        bl.NormQuantBackwardCall(dn, normed.h, normed.rstd, nw.detach(), dweight=torch.empty(k, device=DEV),
                                 want_dweight=False)


# ------------------------------------------------------------------ a step through workspaces

def test_training_step_with_workspaces_in_a_graph(bl, tr):
    """As test_training_step_in_a_graph, at a size whose gradients take the
    operand pass and the norm's a second launch."""
    g = gen(20)
    m, k, n = 600, 600, 600
    assert bl.lib().bitlinear_backward_workspace_bytes(m, n, k, 1, 1) > 0
    x, nw = leaf((m, k), g), leaf((k,), g, torch.float32)
    r, target = (torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    w = [leaf((n, k), g, torch.float32, 0.02) for _ in range(3)]

    def step():
        h, ys = tr.norm_linear(x, w, nw, r)
        z = tr.linear(ys[0], w[1])
        return torch.autograd.grad((*ys[1:], z, h), (x, nw, *w), (target, target, target, r))

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
            x.copy_(torch.randn(m, k, generator=g, device=DEV))
            target.copy_(torch.randn(m, n, generator=g, device=DEV))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i


# ------------------------------------------------------------------ what a call keeps

@pytest.mark.parametrize("residual", [False, True])
def test_norm_linear_checkpoint_size(tr, residual):
    """norm_linear keeps one set of codes for its projections (8 bits an
    activation), 2 bits a weight, 1 / rms a token, and h in bf16: a tensor that
    is there anyway, as the stream with the residual or as x."""
    g = gen(21)
    m, k, ns = 256, 1024, (512, 256, 256)
    x, nw = leaf((m, k), g), leaf((k,), g, torch.float32)
    r = leaf((m, k), g) if residual else None
    ws = [leaf((n, k), g, torch.float32, 0.02) for n in ns]
    kept = {}

    def pack(t):
        kept[t.data_ptr()] = t.numel() * t.element_size()
        return t

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        h, ys = tr.norm_linear(x, ws, nw, r)
    assert kept.pop(h.data_ptr()) == 2 * m * k
    assert kept.pop(nw.data_ptr()) == 4 * k
    assert sum(kept.values()) == m * k + 4 * m + 4 * m + sum(n * k // 4 + 4 for n in ns)


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 8, 16, 17, 100, 520])
@pytest.mark.parametrize("k,ns", [(4096, (4096, 1024, 1024)), (2560, (6912, 6912)), (14336, (4096,)), (2052, (2048, 130))])
def test_grouped_quantized_on_layers(bl, m, k, ns):
    """Projections of layers on one set of codes, in the layouts and plans that
    those sizes take: the grouped forward's bits."""
    g = gen(m)
    x = torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16)
    packs = [bl.pack_weights(0.02 * torch.randn(n, k, generator=g, device=DEV)) for n in ns]
    if k % 256 == 0:
        packs = [(bl.tile_weights(p), s) for p, s in packs]
    biases = [torch.randn(n, generator=g, device=DEV).to(torch.bfloat16) if i else None for i, n in enumerate(ns)]
    residuals = [None if i else torch.randn(m, n, generator=g, device=DEV).to(torch.bfloat16) for i, n in enumerate(ns)]
    ps, ss, count = [p for p, _ in packs], [s for _, s in packs], len(ns)
    want = bl.GroupedCall([x] * count, ps, ss, biases=biases, residuals=residuals)()
    q, xs = bl.act_quant(x)
    kept = q.clone(), xs.clone()
    outs = [torch.empty_like(t) if r is None else r for t, r in zip(want, residuals)]  # added in place
    want = [t.clone() for t in want]
    got = bl.GroupedQuantizedCall([q] * count, [xs] * count, ps, ss, outs, biases=biases, residuals=residuals)()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(q, kept[0]) and torch.equal(xs, kept[1])  # read where they are, and left


def test_input_changed_in_place_is_refused(tr):
    """Without a residual h is x itself: changed before the backward pass, the
    gradient is refused and not made of other values."""
    g = gen(22)
    a, w = leaf((4, 64), g), leaf((24, 64), g, torch.float32, 0.02)
    x = a * 2
    _, (y,) = tr.norm_linear(x, [w])
    x.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.float().sum().backward()
