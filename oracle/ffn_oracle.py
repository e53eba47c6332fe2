"""Plain CPU forms of the operators of a feed-forward block and of a training
step (bitlinear_ffn.h), from their formulas, in float64; roundings that are steps
of a definition are taken where the definition has them.  Shares no code with the
HIP path.

bf16 tensors are uint16 bit patterns, as in bitlinear_oracle.
"""

from __future__ import annotations

import numpy as np

from .bitlinear_oracle import bf16_to_f32, f32_to_bf16


def gated_position(n, k, ktiles, up):
    """(byte offset, shift) of weight [n][k] of the gate (up: False) or the up
    projection in the gated storage."""
    t, r = divmod(k, 256)
    g, i = divmod(r, 64)
    s, e = divmod(i, 16)
    d, j = divmod(e, 4)
    off = ((((n // 16) * ktiles + t) * 2 + int(up)) * 4 + g) * 256 + (n % 16) * 16 + 4 * s + j
    return off, 6 - 2 * d


def gated_pack(ug, uu):
    """Storage bytes (uint8, flat) of ternary weights ug, uu [N, K] (-1, 0, 1)."""
    n, k = ug.shape
    kt = -(-k // 256)
    out = np.zeros(-(-n // 16) * kt * 2048, np.uint8)
    for up, w in ((False, ug), (True, uu)):
        for i in range(n):
            for j in range(k):
                off, sh = gated_position(i, j, kt, up)
                out[off] |= np.uint8((int(w[i, j]) & 3) << sh)
    return out


def activation(act, g):
    """(act(g), act'(g)) in float64."""
    g = np.asarray(g, np.float64)
    if act == "relu2":
        r = np.maximum(g, 0)
        return r * r, 2 * r
    e = np.exp(-np.abs(g))
    s, t = np.where(g >= 0, 1, e) / (1 + e), np.where(g >= 0, e, 1) / (1 + e)  # sigmoid of g and of -g
    return g * s, s * (1 + g * t)


def projection(q, x_scale, u, w_scale):
    """fp32(acc / (x_scale * w_scale)): an exact sum, one fp32 product, one
    division."""
    acc = q.astype(np.float64) @ u.astype(np.float64).T  # integers under 2^53: exact in any order
    d = (x_scale.astype(np.float32)[:, None] * np.float32(w_scale)).astype(np.float32)
    return (acc.astype(np.float32) / d).astype(np.float32)


def gated_forward(q, x_scale, ug, gate_scale, uu, up_scale, act):
    """(a in float64 before its rounding, g fp32, u fp32)."""
    g, u = projection(q, x_scale, ug, gate_scale), projection(q, x_scale, uu, up_scale)
    return activation(act, g)[0] * u.astype(np.float64), g, u


def gate_gradients(da, g, u, act):
    """dg and du as bf16 values (float64), from float64 da, g, u."""
    h, dh = activation(act, g)
    f = np.float32
    return (bf16_to_f32(f32_to_bf16((da * u * dh).astype(f))).astype(np.float64),
            bf16_to_f32(f32_to_bf16((da * h).astype(f))).astype(np.float64))


def gated_backward(da, g, u, act, ug, gate_scale, uu, up_scale, xhat):
    """Gradients in float64, and the sums of their terms' magnitudes."""
    dg, du = gate_gradients(da, g, u, act)
    sg, su = float(gate_scale), float(up_scale)
    ug, uu, xhat = (np.asarray(t, np.float64) for t in (ug, uu, xhat))
    return {"dx": dg @ ug / sg + du @ uu / su, "dx_abs": np.abs(dg) @ np.abs(ug) / sg + np.abs(du) @ np.abs(uu) / su,
            "dw_gate": dg.T @ xhat, "dw_gate_abs": np.abs(dg).T @ np.abs(xhat),
            "dw_up": du.T @ xhat, "dw_up_abs": np.abs(du).T @ np.abs(xhat)}


def w8_position(n, k, ktiles):
    """Offset of weight [n][k] in the 8-bit storage."""
    return (((n // 16) * ktiles + k // 64) * 4 + (k % 64) // 16) * 256 + (n % 16) * 16 + k % 16


def w8_quant(w):
    """(v int8 [N, K], scale fp32 [N]) of fp32 weights."""
    w = w.astype(np.float32)
    s = (np.abs(w).max(axis=1) / np.float32(127)).astype(np.float32)
    s = np.where(s == 0, np.float32(1), s)
    return np.clip(np.rint((w / s[:, None]).astype(np.float32)), -127, 127).astype(np.int8), s


def w8_pack(v):
    """Storage (int8, flat) of v [N, K]."""
    n, k = v.shape
    kt = -(-k // 64)
    out = np.zeros(-(-n // 16) * kt * 1024, np.int8)
    i, j = np.meshgrid(np.arange(n), np.arange(k), indexing="ij")
    out[w8_position(i, j, kt)] = v
    return out


def w8_forward(q, x_scale, v, s):
    """y as bf16 bits: exact sums, one fp32 product and one division, rounded."""
    acc = (q.astype(np.float64) @ v.astype(np.float64).T).astype(np.float32)  # exact, as in projection()
    y = (acc * s.astype(np.float32)).astype(np.float32) / x_scale.astype(np.float32)[:, None]
    return f32_to_bf16(y.astype(np.float32))


def clip(grads, max_norm):
    """(norm, factor) in float64 of fp32 arrays."""
    norm = np.sqrt(sum(np.sum(np.square(g.astype(np.float64))) for g in grads))
    return norm, np.minimum(1.0, max_norm / (norm + 1e-6))
