"""Plain CPU forms of the operators around the BitLinear product, from their
formulas, in float64 (roundings that are steps of an operator's definition are
taken where the definition has them).  Shares no code with the HIP path.

bf16 tensors are uint16 bit patterns, as in bitlinear_oracle.
"""

from __future__ import annotations

import numpy as np

from .bitlinear_oracle import act_quant, add_bf16, bf16_to_f32, f32_to_bf16


def residual_sum(x_bits, r_bits):
    """h = bf16(x + residual); x itself without a residual."""
    return x_bits.copy() if r_bits is None else add_bf16(x_bits, r_bits)


def rms_rstd(h_bits, eps):
    """1 / sqrt(mean(h^2) + eps) per row, float64."""
    h = bf16_to_f32(h_bits).astype(np.float64)
    return 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)


def normed(h_bits, rstd, weight):
    """n = bf16(fp32(h * rstd) * weight) as bits; rstd fp32, weight fp32 or None."""
    n = (bf16_to_f32(h_bits) * np.asarray(rstd, np.float32)[:, None]).astype(np.float32)
    if weight is not None:
        n = (n * np.asarray(weight, np.float32)).astype(np.float32)
    return f32_to_bf16(n)


def rms_norm_quant(x_bits, r_bits, weight, eps, rstd=None):
    """(q, x_scale, h, rstd, n); rstd rounded to fp32, or the given one."""
    h = residual_sum(x_bits, r_bits)
    if rstd is None:
        rstd = rms_rstd(h, eps).astype(np.float32)
    n = normed(h, rstd, weight)
    q, s = act_quant(n)
    return q, s, h, rstd, n


def norm_value(h, weight, eps):
    """The norm without its roundings, on float64 rows (for differences)."""
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return y if weight is None else y * weight


def rms_norm_quant_backward(dn, h, rstd, weight, dh):
    """Gradients of the norm in float64: dx, dweight and, for error bounds, the
    terms they are made of."""
    f = np.float64
    dn, h, r = dn.astype(f), h.astype(f), rstd.astype(f)[:, None]
    g = dn if weight is None else dn * weight.astype(f)
    z = h * r
    c = np.mean(g * z, axis=1, keepdims=True)
    dx = r * (g - z * c)
    if dh is not None:
        dx = dx + dh.astype(f)
    return {"dx": dx, "dweight": (dn * z).sum(0),
            "c_abs": np.mean(np.abs(g * z), axis=1, keepdims=True), "z": z, "g": g, "r": r,
            "dw_abs": np.abs(dn * z).sum(0)}


def restore_activations(q, x_scale):
    """bf16(q / x_scale) as bits: one fp32 division, rounded to bf16."""
    return f32_to_bf16((q.astype(np.float32) / x_scale.astype(np.float32)[:, None]).astype(np.float32))


def w4_position(n, k, ktiles):
    """(byte offset, shift) of weight [n][k] in the 4-bit storage."""
    t, r = divmod(k, 128)
    i, g, j = r // 32, (r % 32) // 8, r % 8
    off = (((n // 16) * ktiles + t) * 4 + g) * 256 + (n % 16) * 16 + 4 * i + j % 4
    return off, 4 if j < 4 else 0


def w4_quant(w, group):
    """(v int8 [N, K], scale bits uint16 [N, K / group]) of fp32 weights."""
    n, k = w.shape
    g = w.astype(np.float32).reshape(n, k // group, group)
    s = f32_to_bf16((np.abs(g).max(axis=2) / np.float32(7)).astype(np.float32))
    s = np.where(s == 0, np.uint16(0x3F80), s).astype(np.uint16)
    v = np.clip(np.rint((g / bf16_to_f32(s)[..., None]).astype(np.float32)), -8, 7)
    return v.reshape(n, k).astype(np.int8), s


def w4_pack(v, s):
    """Storage bytes (codes uint8, scales uint16, flat) of v and scale bits."""
    n, k = v.shape
    groups = s.shape[1]
    nb, kt = -(-n // 16), -(-k // 128)
    codes = np.zeros(nb * kt * 1024, np.uint8)
    scales = np.zeros(nb * groups * 16, np.uint16)
    for i in range(n):
        for j in range(k):
            off, sh = w4_position(i, j, kt)
            codes[off] |= np.uint8((int(v[i, j]) & 15) << sh)
        for g in range(groups):
            scales[((i // 16) * groups + g) * 16 + i % 16] = s[i, g]
    return codes, scales


def w4_forward(q, x_scale, v, s, group):
    """(y float64 before rounding, sum of the terms' magnitudes)."""
    n, k = v.shape
    m = q.shape[0]
    sf = bf16_to_f32(s).astype(np.float64)
    acc = np.einsum("mgi,ngi->mng", q.astype(np.float64).reshape(m, k // group, group),
                    v.astype(np.float64).reshape(n, k // group, group))
    terms = acc * sf[None]
    xs = x_scale.astype(np.float64)[:, None]
    return terms.sum(2) / xs, np.abs(terms).sum(2) / xs
