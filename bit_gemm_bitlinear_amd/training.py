"""Training form of BitLinear: differentiable calls over the library's kernels.

The forward pass ternarizes the latent fp32 weights and quantizes the
activations as the inference path does; the backward pass lets gradients pass
straight through both roundings (the detach() form of the Falcon-Edge blog's
BitLinear).  What is kept between the two is small: the activations as int8
codes with a scale per token, the weights as packed ternary codes; by
norm_linear also 1 / rms per token and h in bf16, which is there anyway (the
residual stream, or x).

    y = linear(x, weight)                                    # one BitLinear
    h, (q, k, v) = norm_linear(x, [wq, wk, wv], norm, residual)  # a block's entry

``norm_linear`` adds the residual, normalizes, quantizes once, and runs every
projection on the same codes.  ``BitLinear`` is ``linear`` as a module.  For
inference pack the trained weights once: ``bitlinear.BitLinear(module.weight)``.

The gradients take up to 2^21 tokens and outputs a layer (bitlinear_backward's
limits).  A gradient of these gradients is not defined (asking for one raises).  To
capture a training step into a HIP graph, drop every eager graph over the same
parameters first, as for any autograd program.
"""

from __future__ import annotations

from typing import Sequence

import torch
from torch.autograd.function import once_differentiable

from . import bitlinear as bl

__all__ = ["BitLinear", "linear", "norm_linear"]


def _aligned(t: torch.Tensor | None):
    """`t` as the kernels take it: contiguous, and copied where it starts off a
    16-byte boundary (a slice of a larger tensor, the gradient that a
    concatenation hands to its parts)."""
    if t is None:
        return None
    t = t.detach().contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _rows(x: torch.Tensor | None):
    return None if x is None else _aligned(x.reshape(-1, x.shape[-1]))


def _check_weights(weights, k):
    """Latent weights [N_i, K] for inputs of `k` columns.  Checked here: a packed
    weight of 16 K columns has the bytes of a tiled one with 16 N rows, and is
    taken for it."""
    for w in weights:
        if w.dim() != 2 or w.shape[1] != k:
            raise ValueError(f"a weight must have shape [N, {k}], got {list(w.shape)}")


def _project(q, x_scale, weights, biases):
    """Packs each latent weight and runs all projections on one set of codes:
    (outputs, packed weights, weight scales)."""
    packs = [bl.pack_weights(_aligned(w)) for w in weights]
    packed, scales = [p for p, _ in packs], [s for _, s in packs]
    count = len(weights)
    ys = bl.GroupedQuantizedCall([q] * count, [x_scale] * count, packed, scales,
                                 biases=[_aligned(b) for b in biases])()
    return ys, packed, scales


def _project_backward(ctx, first, dys, q, x_scale, packed, scales, want_dx):
    """Gradients of the projections' common input (bf16, or None), and per
    projection of its weight and bias; their inputs start at ctx's `first`."""
    dn, dws, dbs = None, [], []
    count = len(dys)
    for i, dy in enumerate(dys):
        want_w, want_b = ctx.needs_input_grad[first + i], ctx.needs_input_grad[first + count + i]
        if dy is None or not (want_dx or want_w or want_b):
            dws.append(None)
            dbs.append(None)
            continue
        dy = _aligned(dy)
        # The kernel's bias sums come with the weights' product: of four columns
        # where the weights' gradient is not wanted.
        codes, dx, dw, db = q if want_w else None, None, None, None
        if want_b and not want_w:
            db = bl.backward_weight(dy, q[:, :4].contiguous(), x_scale, bias=True)[1]
        if want_w or want_dx:
            # Layers that share an input add their gradients up in bf16, rounded
            # after each: what autograd does with a gradient of the input's type.
            dx, dw, sums = bl.BackwardCall(
                dy, codes, x_scale if want_w else None, packed[i] if want_dx else None,
                scales[i] if want_dx else None, bias=want_b and want_w, k=q.shape[1], residual=dn, dx=dn)()
            db = sums if want_w else db
        if want_dx:
            dn = dx
        dws.append(dw)
        dbs.append(db.to(ctx.bias_types[i]) if want_b else None)
    return dn, dws, dbs


class _Linear(torch.autograd.Function):
    """Output rows [M, N], which the caller shapes: of a view made in here,
    autograd refuses in-place operations."""

    @staticmethod
    def forward(ctx, x, weight, bias):
        q, xs = bl.act_quant(_rows(x))
        (y,), packed, scales = _project(q, xs, [weight], [bias])
        ctx.save_for_backward(q, xs, packed[0], scales[0])
        ctx.bias_types = [None if bias is None else bias.dtype]
        ctx.x_shape = x.shape
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        q, xs, packed, scale = ctx.saved_tensors
        dx, (dw,), (db,) = _project_backward(ctx, 1, [dy], q, xs, [packed], [scale],
                                             ctx.needs_input_grad[0])
        return None if dx is None else dx.reshape(ctx.x_shape), dw, db


class _NormLinear(torch.autograd.Function):
    """Rows (see _Linear) of h, with a residual, and of the outputs.  x and the
    residual are not views of rows made outside: they get one gradient tensor,
    which autograd copies for one of two leaves; of two views it would keep
    both, as buffers that share memory."""

    @staticmethod
    def forward(ctx, x, residual, norm_weight, eps, *params):
        count = len(params) // 2
        weights, biases = params[:count], params[count:]
        ctx.set_materialize_grads(False)
        normed = bl.rms_norm_quant(_rows(x), _aligned(norm_weight), _rows(residual), eps)
        ys, packed, scales = _project(normed.q, normed.x_scale, weights, biases)
        ctx.save_for_backward(normed.q, normed.x_scale, normed.h, normed.rstd, norm_weight,
                              *packed, *scales)
        ctx.bias_types = [None if b is None else b.dtype for b in biases]
        ctx.count, ctx.x_shape = count, x.shape
        ctx.has_residual = residual is not None
        return (normed.h, *ys) if residual is not None else tuple(ys)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        q, xs, h, rstd, norm_weight, *rest = ctx.saved_tensors
        packed, scales = rest[:ctx.count], rest[ctx.count:]
        dh, dys = (grads[0], grads[1:]) if ctx.has_residual else (None, grads)
        want_x, want_r, want_norm = ctx.needs_input_grad[:3]
        dn, dws, dbs = _project_backward(ctx, 4, dys, q, xs, packed, scales,
                                         want_x or want_r or want_norm)
        dx = dweight = None
        if dn is not None:
            dx, dweight = bl.rms_norm_quant_backward(dn, h, rstd, _aligned(norm_weight), _aligned(dh),
                                                    want_dweight=want_norm)
            dx = dx.reshape(ctx.x_shape)
            if want_norm:
                dweight = dweight.to(norm_weight.dtype)
        elif dh is not None:  # no projection's output was used
            dx = dh.reshape(ctx.x_shape)
        return (dx if want_x else None, dx if want_r else None, dweight if want_norm else None, None,
                *dws, *dbs)


class _NoTokens(torch.autograd.Function):
    """Output rows [0, N] of each of `widths`, for inputs x without a token:
    every gradient is zero.  (The library's calls take one token or more.)"""

    @staticmethod
    def forward(ctx, widths, x, *params):
        bl._require(x, torch.bfloat16, x.dim(), "x")
        ctx.like = [(t.shape, t.dtype, t.device) if t is not None else None for t in (x, *params)]
        return tuple(x.new_empty((0, n)) for n in widths)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        return None, *(torch.zeros(like[0], dtype=like[1], device=like[2]) if want else None
                       for like, want in zip(ctx.like, ctx.needs_input_grad[1:]))


def linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None) -> torch.Tensor:
    """BitLinear of bf16 x [..., K] on latent fp32 weights [N, K] and an
    optional bf16 bias [N]: bf16 [..., N], differentiable in all three.  Without
    a token (a leading size of 0) y is empty and every gradient zero."""
    _check_weights([weight], x.shape[-1])
    y = _Linear.apply(x, weight, bias) if x.numel() else _NoTokens.apply([weight.shape[0]], x, weight, bias)[0]
    return y.reshape(*x.shape[:-1], weight.shape[0])


def norm_linear(x: torch.Tensor, weights: Sequence[torch.Tensor],
                norm_weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                biases: Sequence[torch.Tensor | None] | None = None, eps: float = 1e-6):
    """RMSNorm of bf16 x [..., K] (plus a residual of the same shape) with an
    optional bf16 or fp32 weight [K], then the BitLinears `weights` (latent
    fp32 [N_i, K], up to 16) of its output.  Returns (h, outputs): h is the sum
    with the residual, what the next residual add takes (x itself without one),
    outputs a list of bf16 [..., N_i]; differentiable throughout.  The backward
    pass needs h: changed in place before it, it is refused there.  Without a
    token everything is empty and every gradient zero, as in linear()."""
    weights = list(weights)
    biases = [None] * len(weights) if biases is None else list(biases)
    if not weights or len(biases) != len(weights):
        raise ValueError("norm_linear: at least one weight, and one bias (or None) for each")
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual must have shape {tuple(x.shape)}, got {tuple(residual.shape)}")
    _check_weights(weights, x.shape[-1])
    if x.numel():
        out = _NormLinear.apply(x, residual, norm_weight, eps, *weights, *biases)
    else:
        widths = [w.shape[0] for w in weights]
        out = _NoTokens.apply(widths if residual is None else [x.shape[-1], *widths], x, residual, norm_weight,
                              *weights, *biases)
    h, out = (x, out) if residual is None else (out[0].reshape(x.shape), out[1:])
    return h, [y.reshape(*x.shape[:-1], y.shape[1]) for y in out]


class BitLinear(torch.nn.Module):
    """A trainable BitLinear: latent fp32 weight [out, in], optional bf16
    bias."""

    def __init__(self, in_features: int, out_features: int, bias: bool = False, device=None):
        super().__init__()
        self.in_features, self.out_features = in_features, out_features
        self.weight = torch.nn.Parameter(
            torch.randn(out_features, in_features, dtype=torch.float32, device=device) * in_features ** -0.5)
        self.bias = (torch.nn.Parameter(torch.zeros(out_features, dtype=torch.bfloat16, device=device))
                     if bias else None)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return linear(x, self.weight, self.bias)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, bias={self.bias is not None}"
