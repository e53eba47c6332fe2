"""Operators around the BitLinear product, as cases to measure.

Three operators (and the gradients of two of them), each in its plain form
(elementary torch operations in fp32, in 64 bits where a rounding border or a
long sum asks for it) and through the package's own calls (`own`):

  norm           residual add, RMSNorm, per-token int8 codes and scale
  norm_backward  gradients of the norm: its input (and the residual), its weight
  backward       gradients of BitLinear from its 8-bit activation checkpoint
                 (codes and scales) and its packed ternary weights
  w4             product of int8 activations with 4-bit weights, group scales

Definitions (all rounding steps are part of the operator and the same in
every form):

  h      = bf16(x + residual)                     (h = x without a residual)
  rstd   = fp32(1 / sqrt(mean(h^2) + eps))        mean and root in 64 bits
  n      = bf16(fp32(h * rstd) * weight)          two fp32 products
  xs     = 127 / max(max|n|, 1e-5),  q = clamp(round_half_even(n * xs), -128, 127)
  xhat   = bf16(q / xs)                           the restored activation
  norm_backward: g = dn * weight, z = h * rstd,
           dx = bf16(rstd * (g - z * mean(g * z)) + dh),  dweight = sum_m dn * z
  backward: dx = bf16((dy . u) / w_scale), dw = dy^T . xhat, db = sum_m dy
  w4     : y = bf16(sum_g scale[n, g] * (sum_{k in g} q[m, k] * v[n, k]) / xs[m])
"""

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # one new token: the norm before the projections of an 8B-class layer
        {"name": "norm_m1_k4096", "op": "norm", "m": 1, "k": 4096, "residual": True, "weight": "bf16"},
        # a prompt through a 2B-class layer
        {"name": "norm_m2048_k2560", "op": "norm", "m": 2048, "k": 2560, "residual": True, "weight": "bf16"},
        # the norm before the down projection of an 8B-class layer (no residual),
        # a ragged batch, weights kept in fp32 for training
        {"name": "norm_m777_k14332", "op": "norm", "m": 777, "k": 14332, "residual": False, "weight": "fp32"},
        # training: gradients of the norm, a short and a long batch of tokens
        {"name": "norm_backward_m512_k4096", "op": "norm_backward", "m": 512, "k": 4096, "dh": True, "weight": "bf16"},
        {"name": "norm_backward_m8191_k2560", "op": "norm_backward", "m": 8191, "k": 2560, "dh": True, "weight": "fp32"},
        # training: gradients of one projection -- 2B-class gate/up, 8B-class
        # down, a small ragged one with a bias, and a short fine-tuning batch
        {"name": "backward_m2048_n6912_k2560", "op": "backward", "m": 2048, "n": 6912, "k": 2560, "bias": False},
        {"name": "backward_m2048_n4096_k14336", "op": "backward", "m": 2048, "n": 4096, "k": 14336, "bias": False},
        {"name": "backward_m301_n1001_k1284", "op": "backward", "m": 301, "n": 1001, "k": 1284, "bias": True},
        {"name": "backward_m40_n4096_k4096", "op": "backward", "m": 40, "n": 4096, "k": 4096, "bias": False},
        # serving: the 4-bit output head and projections -- one token through an
        # 8B-class gate/up, a batch of 16 through a head of 32768 outputs, and
        # a few tokens through a ragged one with short groups
        {"name": "w4_m1_n14336_k4096", "op": "w4", "m": 1, "n": 14336, "k": 4096, "group": 128},
        {"name": "w4_m16_n32768_k4096", "op": "w4", "m": 16, "n": 32768, "k": 4096, "group": 64},
        {"name": "w4_m5_n1003_k2080", "op": "w4", "m": 5, "n": 1003, "k": 2080, "group": 32},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "backward", "w4"])
    if op == "norm":
        k = 4 * _log(rng, 16, 3584)
        m = min(_log(rng, 1, 4096), 11_000_000 // k)
        return {"op": op, "m": m, "k": k, "residual": rng.random() < 0.6,
                "weight": rng.choice(["bf16", "fp32", "none"])}
    if op == "norm_backward":
        k = 4 * _log(rng, 16, 3584)
        m = min(_log(rng, 1, 8192), 20_000_000 // k)
        return {"op": op, "m": m, "k": k, "dh": rng.random() < 0.6,
                "weight": rng.choice(["bf16", "fp32", "none"])}
    if op == "backward":
        n, k = _log(rng, 16, 14336), 4 * _log(rng, 16, 3584)
        m = max(1, min(_log(rng, 1, 2048), 100_000_000_000 // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k, "bias": rng.random() < 0.3}
    group = rng.choice([32, 64, 128])
    k = group * _log(rng, 2, 8192 // group)
    n = min(_log(rng, 16, 32768), 134_000_000 // k)
    return {"op": op, "m": rng.randint(1, 16), "n": n, "k": k, "group": group}


# ---------------------------------------------------------------- inputs

def _div32(a, b):
    """fp32 quotient, correctly rounded (a 64-bit quotient rounded to fp32 is)."""
    return (a.double() / b.double()).float()


def _quant(n):
    """int8 codes (as fp32 values) and scales of bf16 rows."""
    n32 = n.float()
    xs = _div32(torch.full_like(n32[:, 0], 127.0), n32.abs().amax(1).clamp_min(1e-5))
    return torch.round(n32 * xs[:, None]).clamp_(-128, 127), xs


def _weight(kind, k, gen, dev):
    if kind == "none":
        return None
    w = 1.0 + 0.2 * torch.randn(k, generator=gen, device=dev)
    return w.to(torch.bfloat16) if kind == "bf16" else w


def _stream(m, k, gen, dev):
    """Rows of a residual stream: N(0, 1), 1% of the channels 20 times larger,
    and a padded (all-zero) row now and then."""
    x = torch.randn(m, k, generator=gen, device=dev)
    x *= torch.where(torch.rand(k, generator=gen, device=dev) < 0.01, 20.0, 1.0)
    if m > 1:
        x *= (torch.rand(m, 1, generator=gen, device=dev) > 0.01).float()
    return x


def _grad(m, n, gen, dev):
    """Rows of an output gradient: small, a spread of sizes by token, and zero
    rows where the loss is masked."""
    d = torch.randn(m, n, generator=gen, device=dev) * 1e-3
    d *= torch.exp(torch.randn(m, 1, generator=gen, device=dev))
    if m > 1:
        d *= (torch.rand(m, 1, generator=gen, device=dev) > 0.05).float()
    return d.to(torch.bfloat16)


def _pack_ternary(w):
    """Packed ternary weights [N, K/4] (code u + 1, two bits, first weight in
    the low bits) and the scale 1 / mean|w|."""
    ws = (1.0 / w.double().abs().mean().clamp_min(1e-5)).float().reshape(1)
    c = (torch.round(w * ws).clamp_(-1, 1) + 1).to(torch.uint8)
    c = c.reshape(w.shape[0], -1, 4)
    return c[..., 0] | (c[..., 1] << 2) | (c[..., 2] << 4) | (c[..., 3] << 6), ws


def _pack_w4(w, group):
    """4-bit weights of w [N, K] in the package's storage: values v = -8..7 as
    4-bit two's complement; N padded to whole blocks of 16 rows and K to whole
    tiles of 128 (zeros).  codes [N/16, K/128, 4 (g), 16 (row), 16 (bytes)]:
    byte 4 i + j of row r, lane group g, holds k = 128 t + 32 i + 8 g + j in
    its high four bits and k + 4 in its low four bits.  scales bf16
    [N/16, K/group, 16]."""
    n, k = w.shape
    nb, kt = -(-n // 16), -(-k // 128)
    amax = w.reshape(n, k // group, group).abs().amax(2)
    s = (amax / 7).to(torch.bfloat16)
    s = torch.where(s == 0, torch.ones_like(s), s)
    v = torch.round(w.reshape(n, k // group, group) / s.float()[..., None]).clamp_(-8, 7)
    full = torch.zeros(nb * 16, kt * 128, dtype=torch.int8, device=w.device)
    full[:n, :k] = v.reshape(n, k).to(torch.int8)
    b = (full.to(torch.int16) & 15).to(torch.uint8).reshape(nb, 16, kt, 4, 4, 2, 4)  # row, t, i, g, half, j
    b = (b[..., 0, :] << 4) | b[..., 1, :]
    codes = b.permute(0, 2, 4, 1, 3, 5).contiguous().reshape(nb, kt, 4, 16, 16)
    sc = torch.zeros(nb * 16, k // group, dtype=torch.bfloat16, device=w.device)
    sc[:n] = s
    return codes, sc.reshape(nb, 16, k // group).permute(0, 2, 1).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    op, m, k = case["op"], case["m"], case["k"]
    st = {"op": op}
    if op == "norm":
        st["x"] = _stream(m, k, gen, dev).to(torch.bfloat16)
        st["residual"] = (3 * torch.randn(m, k, generator=gen, device=dev)).to(torch.bfloat16) if case["residual"] else None
        st["weight"] = _weight(case["weight"], k, gen, dev)
    elif op == "norm_backward":
        st["h"] = _stream(m, k, gen, dev).to(torch.bfloat16)
        st["rstd"] = (1.0 / torch.sqrt(st["h"].double().square().mean(1) + EPS)).float()
        st["dn"] = _grad(m, k, gen, dev)
        st["dh"] = _grad(m, k, gen, dev) if case["dh"] else None
        st["weight"] = _weight(case["weight"], k, gen, dev)
    elif op == "backward":
        n = case["n"]
        q, st["x_scale"] = _quant(_stream(m, k, gen, dev).to(torch.bfloat16))
        st["q"] = q.to(torch.int8)
        st["packed"], st["w_scale"] = _pack_ternary(0.02 * torch.randn(n, k, generator=gen, device=dev))
        st["dy"] = _grad(m, n, gen, dev)
        st["bias"] = case["bias"]
    else:
        n = case["n"]
        q, st["x_scale"] = _quant(_stream(m, k, gen, dev).to(torch.bfloat16))
        st["q"] = q.to(torch.int8)
        st["codes"], st["scales"] = _pack_w4(0.02 * torch.randn(n, k, generator=gen, device=dev), case["group"])
        st["n"], st["group"] = n, case["group"]
    if own:  # the prepared call a program keeps beside its buffers
        from bit_gemm_bitlinear_amd import bitlinear as bl

        if op == "norm":
            st["call"] = bl.NormQuantCall(st["x"], st["weight"], st["residual"], eps=EPS)
            st["xhat"] = torch.empty_like(st["x"])
        elif op == "norm_backward":
            st["call"] = bl.NormQuantBackwardCall(st["dn"], st["h"], st["rstd"], st["weight"], st["dh"])
        elif op == "backward":
            st["call"] = bl.BackwardCall(st["dy"], st["q"], st["x_scale"], st["packed"], st["w_scale"], bias=st["bias"])
        else:
            st["call"] = bl.W4Call(st["q"], st["x_scale"], bl.W4Weights(st["codes"], st["scales"], n, k, st["group"]))
    return st


# ---------------------------------------------------------------- one pass

def _unpack_ternary(packed):
    p = packed[..., None] >> torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=packed.device)
    return (p & 3).reshape(packed.shape[0], -1).float() - 1.0


def _unpack_w4(codes, scales, n, k, group):
    nb, kt = codes.shape[:2]
    hi, lo = (codes >> 4).to(torch.int32), (codes & 15).to(torch.int32)
    v = torch.stack([hi, lo], -1).reshape(nb, kt, 4, 16, 4, 4, 2)  # g, row, i, j, half
    v = v.permute(0, 3, 1, 4, 2, 6, 5).reshape(nb * 16, kt * 128)[:n, :k]
    v = (v - 16 * (v > 7)).float()
    s = scales.float().permute(0, 2, 1).reshape(nb * 16, -1)[:n]
    return (v.reshape(n, k // group, group) * s[..., None]).reshape(n, k)


def _plain(st):
    op = st["op"]
    if op == "norm":
        # h is an output in bf16 and the norm is that of h; the codes are those
        # of the norm's bf16 output.  The mean of squares in 64 bits: a
        # different last bit of rstd moves codes next to a rounding border.
        h = st["x"] if st["residual"] is None else (st["x"].float() + st["residual"].float()).to(torch.bfloat16)
        h32 = h.float()
        rstd = (1.0 / torch.sqrt(h32.double().square().mean(1) + EPS)).float()
        n = h32 * rstd[:, None]
        if st["weight"] is not None:
            n = n * st["weight"].float()
        q, xs = _quant(n.to(torch.bfloat16))
        return {"h": h, "rstd": rstd, "x_scale": xs, "xhat": _div32(q, xs[:, None]).to(torch.bfloat16)}
    if op == "norm_backward":
        dn, z = st["dn"].float(), st["h"].float() * st["rstd"][:, None]
        g = dn if st["weight"] is None else dn * st["weight"].float()
        dx = st["rstd"][:, None] * (g - z * (g * z).mean(1, keepdim=True))
        if st["dh"] is not None:
            dx = dx + st["dh"].float()
        out = {"dx": dx.to(torch.bfloat16)}
        if st["weight"] is not None:
            out["dweight"] = (dn * z).sum(0)
        return out
    if op == "backward":
        dy = st["dy"].float()
        xhat = _div32(st["q"].float(), st["x_scale"][:, None]).to(torch.bfloat16).float()
        out = {"dx": ((dy @ _unpack_ternary(st["packed"])) / st["w_scale"]).to(torch.bfloat16),
               "dw": dy.t() @ xhat}
        if st["bias"]:
            out["db"] = dy.sum(0)
        return out
    w = _unpack_w4(st["codes"], st["scales"], st["n"], st["q"].shape[1], st["group"])
    return {"y": ((st["q"].float() @ w.t()) / st["x_scale"][:, None]).to(torch.bfloat16)}


def run(state):
    if not own:
        return _plain(state)
    op = state["op"]
    if op == "norm":
        from bit_gemm_bitlinear_amd import bitlinear as bl

        r = state["call"]()
        return {"h": r.h, "rstd": r.rstd, "x_scale": r.x_scale,
                "xhat": bl.restore_activations(r.q, r.x_scale, out=state["xhat"])}
    if op == "norm_backward":
        dx, dweight = state["call"]()
        return {"dx": dx} if dweight is None else {"dx": dx, "dweight": dweight}
    if op == "backward":
        dx, dw, db = state["call"]()
        return {"dx": dx, "dw": dw} if db is None else {"dx": dx, "dw": dw, "db": db}
    return {"y": state["call"]()}


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    wb = {"bf16": 2, "fp32": 4, "none": 0}.get(case.get("weight"), 0) * k
    if op == "norm":
        # x (and the residual) in, h out where there is a residual, the codes
        # written and read back, the restored activations, two row statistics
        return {"bytes": m * k * ((2 + 2 + 2 if case["residual"] else 2) + 1 + 1 + 2) + wb + 12 * m,
                "flops": 10 * m * k}
    if op == "norm_backward":
        return {"bytes": m * k * (2 + 2 + 2 + (2 if case["dh"] else 0)) + 4 * m + wb + (4 * k if wb else 0),
                "flops": 10 * m * k}
    if op == "backward":
        n = case["n"]
        return {"bytes": 2 * m * n + m * k + 4 * m + n * k // 4 + 2 * m * k + 4 * n * k + (4 * n if case["bias"] else 0),
                "flops": 4 * m * n * k}
    n, group = case["n"], case["group"]
    return {"bytes": n * k // 2 + 2 * n * (k // group) + m * k + 4 * m + 2 * m * n, "flops": 2 * m * n * k}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The outputs from the definition, in 64 bits; a rounding that is a step
    of the definition (h, rstd, n, the codes, xhat) is taken there, and a
    product of two fp32 values is exact in 64 bits before it."""
    st = prepare(case, seed)
    op, f = case["op"], torch.float64
    if op == "norm":
        h = st["x"].to(f)
        if st["residual"] is not None:
            h = (h + st["residual"].to(f)).float().to(torch.bfloat16).to(f)
        rstd = torch.rsqrt((h * h).sum(-1, keepdim=True) / h.shape[1] + EPS)
        z = (h * rstd.float().to(f)).float().to(f)
        if st["weight"] is not None:
            z = (z * st["weight"].to(f)).float().to(f)
        z = z.float().to(torch.bfloat16).to(f)
        xs = 127.0 / torch.clamp(z.abs().max(dim=-1, keepdim=True).values, min=float(torch.tensor(1e-5)))
        s32 = xs.float().to(f)
        q = torch.clamp(torch.round((z * s32).float().to(f)), -128, 127)
        return {"h": h, "rstd": rstd[:, 0], "x_scale": xs[:, 0], "xhat": q / s32}
    if op == "norm_backward":
        h, dn, r = st["h"].to(f), st["dn"].to(f), st["rstd"].to(f)[:, None]
        w = torch.ones(h.shape[1], dtype=f, device=h.device) if st["weight"] is None else st["weight"].to(f)
        k = h.shape[1]
        dot = torch.sum(dn * w * h, dim=1, keepdim=True)
        dx = r * w * dn - (r ** 3 / k) * dot * h
        if st["dh"] is not None:
            dx = dx + st["dh"].to(f)
        return {"dx": dx} if st["weight"] is None else {"dx": dx, "dweight": torch.sum(dn * (h * r), dim=0)}
    if op == "backward":
        dy = st["dy"].to(f)
        xhat = (st["q"].to(f) / st["x_scale"].to(f).unsqueeze(1)).float().to(torch.bfloat16).to(f)
        p = st["packed"].to(torch.int32)
        u = torch.stack([((p // 4 ** i) % 4) - 1 for i in range(4)], dim=2).flatten(1).to(f)
        out = {"dx": torch.mm(dy, u) / st["w_scale"].to(f), "dw": torch.mm(dy.t().contiguous(), xhat)}
        if st["bias"]:
            out["db"] = torch.sum(dy, dim=0)
        return out
    # each weight looked up at its own place in the storage
    n, k, group = case["n"], case["k"], case["group"]
    kk = torch.arange(k, device=st["q"].device)
    t, i, g, j = kk // 128, kk % 128 // 32, kk % 32 // 8, kk % 8
    rows = torch.arange(n, device=kk.device)[:, None]
    byte = st["codes"][rows // 16, t, g, rows % 16, 4 * i + j % 4].to(torch.int32)
    v = torch.where(j < 4, byte // 16, byte % 16)
    v = torch.where(v >= 8, v - 16, v).to(f) * st["scales"][rows // 16, kk // group, rows % 16].to(f)
    return {"y": torch.mm(st["q"].to(f), v.t().contiguous()) / st["x_scale"].to(f)[:, None]}
