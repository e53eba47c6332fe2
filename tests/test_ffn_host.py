"""Host-side checks of the operators of a feed-forward block and of a training
step (bitlinear_ffn.h) that need no GPU: exports, refusals (every call below
fails validation, so no kernel is launched), the oracle's formulas against
differences, and the storages against their descriptions."""

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import oracle
from oracle import ffn as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, ESHAPE, EALIGN, EWORKSPACE = 0, 1, 2, 3, 4
P = ctypes.c_void_p
A = [P(0x1000000000 * (i + 1)) for i in range(14)]  # aligned, far apart, never dereferenced
ODD = P(0x1000000008)
BIG = ctypes.c_size_t(1 << 60)


@pytest.fixture(scope="module")
def bl():
    from bit_gemm_bitlinear_amd import build as b

    if not os.path.exists(b.LIB):
        b.build()
    from bit_gemm_bitlinear_amd import bitlinear

    return bitlinear


@pytest.fixture(scope="module")
def lib(bl):
    return bl.lib()


def test_exports(bl):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "bitlinear_ffn.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(bitlinear_\w+)\s*\(", text)))
    assert len(names) == 14
    out = subprocess.run(["nm", "-D", "--defined-only", bl.LIB_PATH], capture_output=True, text=True).stdout
    assert set(names) <= set(re.findall(r"\bT (bitlinear_\w+)", out))
    assert set(names) <= set(bl._SIGS)


BAD = [(0, 8, 64), (2, 0, 64), (2, 8, 0), (2, 8, 66), (2, 8, 2 ** 17 + 4), (2, 2 ** 24 + 1, 64), (2 ** 19 + 1, 8, 64),
       (-1, 8, 64), (2 ** 19, 2 ** 18 + 1, 64)]


# ---------------------------------------------------------------- gated

def gated(lib, m=20, n=40, k=68, q=A[0], xs=A[1], codes=A[2], sg=A[3], su=A[4], act=1, a=A[5], g=None, u=None, ws=A[8],
          size=BIG):
    return lib.bitlinear_gated_forward(m, n, k, q, xs, codes, sg, su, act, a, g, u, ws, size, None)


def test_gated_refusals(lib):
    for m, n, k in BAD:
        assert gated(lib, m, n, k) == ESHAPE, (m, n, k)
        assert lib.bitlinear_gated_forward_workspace_bytes(m, n, k) == 0
    for name in ("q", "xs", "codes", "sg", "su", "a"):
        assert gated(lib, **{name: None}) == EINVAL, name
        assert gated(lib, **{name: ODD}) == EALIGN, name
    assert gated(lib, g=ODD, u=A[7]) == EALIGN and gated(lib, ws=ODD) == EALIGN
    for act in (0, 3, -1):
        assert gated(lib, act=act) == EINVAL
    assert gated(lib, g=A[6]) == EINVAL and gated(lib, u=A[6]) == EINVAL  # kept together
    for bad in (dict(a=A[0]), dict(a=A[1]), dict(a=A[2]), dict(a=A[3]), dict(g=A[5], u=A[7]), dict(g=A[6], u=A[6]),
                dict(g=A[0], u=A[7])):
        assert gated(lib, **bad) == EINVAL, bad
    need = lib.bitlinear_gated_forward_workspace_bytes(20, 40, 68)
    if need:
        assert gated(lib, size=need - 1) == EWORKSPACE and gated(lib, ws=None) == EWORKSPACE
        assert gated(lib, ws=A[5]) == EINVAL and gated(lib, ws=A[0]) == EINVAL


def test_gated_weights_refusals(lib):
    def call(n=32, k=256, gate=A[0], lg=0, up=A[1], lu=1, codes=A[2]):
        return lib.bitlinear_gated_weights(n, k, gate, lg, up, lu, codes, None)

    for _, n, k in BAD[1:6]:
        assert call(n, k, lu=0) == ESHAPE
        assert lib.bitlinear_gated_weights_bytes(n, k) == 0
    assert call(lg=2) == EINVAL and call(lu=-1) == EINVAL
    assert call(n=17) == ESHAPE and call(k=260) == ESHAPE  # the tiled layout
    for name in ("gate", "up", "codes"):
        assert call(**{name: None}) == EINVAL and call(**{name: ODD}) == EALIGN
    assert call(codes=A[0]) == EINVAL and call(codes=A[1]) == EINVAL
    assert lib.bitlinear_gated_weights_bytes(17, 260) == 2 * 2 * 2048


def gback(lib, m=20, n=40, k=68, act=1, da=A[0], g=A[1], u=A[2], gate=A[3], lg=0, up=A[4], lu=0, sg=A[5], su=A[6],
          res=None, dx=A[7], q=A[8], xs=A[9], dwg=A[10], dwu=A[11], acc=0, ws=A[12], size=BIG):
    return lib.bitlinear_gated_backward(m, n, k, act, da, g, u, gate, lg, up, lu, sg, su, res, dx, q, xs, dwg, dwu, acc,
                                        ws, size, None)


def test_gated_backward_refusals(lib):
    bytes_ = lib.bitlinear_gated_backward_workspace_bytes
    for m, n, k in ((0, 8, 64), (2, 0, 64), (2, 8, 66), (2 ** 21 + 1, 8, 64), (2, 2 ** 20 + 1, 64), (2, 2 ** 62, 64)):
        assert gback(lib, m, n, k) == ESHAPE, (m, n, k)
        assert bytes_(m, n, k, 1, 1) == 0
    assert bytes_(20, 40, 68, 0, 0) == 0
    for name in ("da", "g", "u", "gate", "up", "sg", "su", "q", "xs"):
        assert gback(lib, **{name: None}) == EINVAL, name
        assert gback(lib, **{name: ODD}) == EALIGN, name
    for name in ("dx", "dwg", "dwu", "res", "ws"):
        assert gback(lib, **{name: ODD}) == EALIGN, name
    for bad in (dict(act=0), dict(act=3), dict(acc=2), dict(lg=2), dict(lu=-1), dict(dwg=None), dict(dwu=None),
                dict(dx=None, dwg=None, dwu=None), dict(dx=None, res=A[13])):
        assert gback(lib, **bad) == EINVAL, bad
    assert gback(lib, lg=1) == ESHAPE  # tiled weights of 40 x 68
    need = bytes_(20, 40, 68, 1, 1)
    assert need > 0 and gback(lib, size=need - 1) == EWORKSPACE and gback(lib, ws=None) == EWORKSPACE
    for bad in (dict(dx=A[0]), dict(dx=A[1]), dict(dx=A[3]), dict(dwg=A[8]), dict(dwg=A[11]), dict(ws=A[2]),
                dict(ws=A[7]), dict(res=A[10]), dict(res=P(A[7].value + 16)), dict(dwu=A[9])):
        assert gback(lib, **bad) == EINVAL, bad


def test_gated_storage_position():
    """Every weight at a place of its own, and the places the header names."""
    seen = set()
    for up in (False, True):
        for n in range(17):
            for k in range(260):
                seen.add(ref.gated_position(n, k, 2, up))
    assert len(seen) == 2 * 17 * 260
    assert ref.gated_position(0, 0, 1, False) == (0, 6) and ref.gated_position(0, 4, 1, False) == (0, 4)
    assert ref.gated_position(0, 1, 1, True) == (1025, 6) and ref.gated_position(3, 64 + 17, 1, False) == (256 + 48 + 5, 6)
    assert ref.gated_position(16, 256, 2, False) == (6144, 6)


@pytest.mark.parametrize("act", ["relu2", "silu"])
def test_gate_gradients_against_differences(act):
    rng = np.random.default_rng(1)
    g, u = rng.standard_normal(2000) * 3, rng.standard_normal(2000)
    g = np.concatenate([g, [0.0, -0.0, 1e-3, -1e-3, 40.0, -40.0, 100.0, -100.0]])
    u = np.concatenate([u, np.ones(8)])
    h, dh = ref.activation(act, g)
    t = 1e-6 * np.maximum(1, np.abs(g))
    num = (ref.activation(act, g + t)[0] - ref.activation(act, g - t)[0]) / (2 * t)
    # third derivatives are at most 1 (silu); relu2 has a kink of its second
    assert np.allclose(num, dh, rtol=1e-6, atol=2e-6)
    # the two gradients are those of act(g) * u before they are rounded to bf16
    da = rng.standard_normal(g.shape)
    dg, du = ref.gate_gradients(da, g, u, act)
    assert np.all(np.abs(dg - da * u * dh) <= 2.0 ** -8 * np.abs(da * u * dh) * (1 + 1e-6) + 1e-38)
    assert np.all(np.abs(du - da * h) <= 2.0 ** -8 * np.abs(da * h) * (1 + 1e-6) + 1e-38)


# ------------------------------------------------------------------- w8

def w8(lib, m=20, n=40, k=68, q=A[0], xs=A[1], codes=A[2], s=A[3], b=A[4], y=A[5], ws=A[6], size=BIG):
    return lib.bitlinear_w8_forward(m, n, k, q, xs, codes, s, b, y, ws, size, None)


def test_w8_refusals(lib):
    for m, n, k in BAD:
        assert w8(lib, m, n, k) == ESHAPE, (m, n, k)
        assert lib.bitlinear_w8_forward_workspace_bytes(m, n, k) == 0
    for name in ("q", "xs", "codes", "s", "y"):
        assert w8(lib, **{name: None}) == EINVAL, name
    for name in ("q", "xs", "codes", "s", "y", "b", "ws"):
        assert w8(lib, **{name: ODD}) == EALIGN, name
    for bad in (dict(y=A[0]), dict(y=A[1]), dict(y=A[2]), dict(y=A[3]), dict(y=A[4])):
        assert w8(lib, **bad) == EINVAL, bad
    need = lib.bitlinear_w8_forward_workspace_bytes(20, 40, 68)
    if need:
        assert w8(lib, size=need - 1) == EWORKSPACE and w8(lib, ws=None) == EWORKSPACE
        assert w8(lib, ws=A[5]) == EINVAL and w8(lib, ws=A[2]) == EINVAL
    for n, k in ((0, 64), (8, 66), (8, 2 ** 17 + 4), (2 ** 24 + 1, 64)):
        assert lib.bitlinear_w8_pack(A[0], n, k, A[1], A[2], None) == ESHAPE
        assert lib.bitlinear_w8_unpack(A[0], A[1], n, k, A[2], None) == ESHAPE
        assert lib.bitlinear_w8_codes_bytes(n, k) == 0
    assert lib.bitlinear_w8_codes_bytes(17, 68) == 2 * 2 * 1024
    assert lib.bitlinear_w8_pack(A[0], 8, 64, A[0], A[2], None) == EINVAL
    assert lib.bitlinear_w8_pack(A[0], 8, 64, A[1], A[1], None) == EINVAL
    assert lib.bitlinear_w8_pack(ODD, 8, 64, A[1], A[2], None) == EALIGN
    assert lib.bitlinear_w8_unpack(A[0], A[1], 8, 64, A[0], None) == EINVAL
    assert lib.bitlinear_w8_unpack(None, A[1], 8, 64, A[2], None) == EINVAL


def test_w8_sums_fit_int32():
    # the longest K and the largest codes of both sides
    assert 128 * 127 * 2 ** 17 < 2 ** 31 and 127 * 64 * 2 ** 17 < 2 ** 31


# ----------------------------------------------------------------- clip

def grads(bl, *items):
    arr = (bl.Gradient * max(1, len(items)))()
    for i, (g, o, n, t) in enumerate(items):
        arr[i] = bl.Gradient(g, o, n, t, 0)
    return arr


def test_clip_refusals(bl, lib):
    a = [p.value for p in A]

    def clip(arr, max_norm=1.0, norm=A[10], ws=A[11], size=BIG, count=None):
        n = len(arr) if count is None else count
        return lib.bitlinear_clip_gradients(n, arr, max_norm, norm, ws, size, None)

    def norm_only(arr, norm=A[10], ws=A[11], size=BIG, count=None):
        return lib.bitlinear_grad_norm(len(arr) if count is None else count, arr, norm, ws, size, None)

    one = grads(bl, (a[0], a[1], 100, 2))
    for call in (clip, norm_only):
        assert call(one, count=0) == EINVAL and call(one, count=-1) == EINVAL and call(one, count=2 ** 20 + 1) == EINVAL
        assert call(None, count=1) == EINVAL
        assert call(one, norm=None) == EINVAL and call(one, norm=ODD) == EALIGN
        assert call(one, ws=None) == EWORKSPACE and call(one, size=7) == EWORKSPACE and call(one, ws=ODD) == EALIGN
        assert call(grads(bl, (a[0], a[1], -1, 2))) == ESHAPE
        assert call(grads(bl, (a[0], a[1], 2 ** 40 + 1, 2))) == ESHAPE
        assert call(grads(bl, (a[0], a[1], 2 ** 39, 1), (a[2], a[3], 2 ** 39 + 1, 1))) == ESHAPE
        for t in (0, 3, -1):
            assert call(grads(bl, (a[0], a[1], 100, t))) == EINVAL
        assert call(grads(bl, (0, a[1], 100, 2))) == EINVAL
        assert call(grads(bl, (a[0] + 2, a[1], 100, 2))) == EALIGN
        assert call(grads(bl, (a[0] + 1, a[1], 100, 1))) == EALIGN
        assert call(one, norm=P(a[0] + 16)) == EINVAL and call(one, ws=P(a[0])) == EINVAL
        assert call(one, norm=A[11]) == EINVAL
        bad = grads(bl, (a[0], a[1], 100, 2))
        bad[0].reserved = 1
        assert call(bad) == EINVAL
    assert clip(grads(bl, (a[0], 0, 100, 2))) == EINVAL
    for m in (-1.0, float("nan"), -0.5):
        assert clip(one, max_norm=m) == EINVAL
    # overlaps: an output is its own gradient exactly, or apart from everything
    for arr in (grads(bl, (a[0], a[0] + 16, 100, 2)), grads(bl, (a[0], a[0], 100, 2), (a[0], a[0], 100, 2)),
                grads(bl, (a[0], a[1], 100, 2), (a[2], a[1] + 396, 100, 2)),
                grads(bl, (a[0], a[1], 100, 2), (a[1], a[2], 100, 2)),
                grads(bl, (a[0], a[0], 100, 2), (a[0] + 200, a[2], 10, 2)),
                grads(bl, (a[0], a[3], 1000, 2), (a[0] + 100, a[0] + 100, 4, 2))):
        assert clip(arr) == EINVAL
    assert lib.bitlinear_grad_norm_workspace_bytes(1, one) >= 8
    assert lib.bitlinear_grad_norm_workspace_bytes(0, one) == 0
    assert lib.bitlinear_grad_norm_workspace_bytes(1, grads(bl, (0, 0, -1, 2))) == 0


def test_binding_refusals(bl):
    t = torch.zeros(4, 64, dtype=torch.int8)
    with pytest.raises(TypeError):
        bl.forward_w8(t, None, None)
    with pytest.raises(TypeError):
        bl.pack_weights_w8(torch.zeros(4, 64))
    with pytest.raises(TypeError):
        bl.clip_grads([torch.zeros(4)], 1.0)
    with pytest.raises(ValueError):
        bl.clip_grads([], 1.0)
    for m in (-1.0, float("nan")):
        with pytest.raises(ValueError):
            bl.clip_grads([torch.zeros(4)], m)
    with pytest.raises(ValueError):
        bl._activation("gelu")
    for shape, stride, dense in (((4, 6), (6, 1), True), ((4, 6), (1, 4), True), ((4, 6), (7, 1), False),
                                 ((4, 6), (0, 1), False), ((4, 1), (1, 9), True), ((0, 5), (5, 1), True),
                                 ((2, 3, 4), (4, 8, 1), True), ((5,), (2,), False), ((), (), True)):
        x = torch.zeros(100).as_strided(shape, stride)
        assert bl._dense(x) == dense, (shape, stride)


def test_training_refusals():
    from bit_gemm_bitlinear_amd import training as tr

    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(8, 64)
    with pytest.raises(ValueError):
        tr.norm_gated(x, w, w, activation="tanh")
    with pytest.raises(ValueError):
        tr.norm_gated(x, w, torch.zeros(9, 64))
    with pytest.raises(ValueError):
        tr.norm_gated(x, w, torch.zeros(8, 68))
    with pytest.raises(ValueError):
        tr.norm_gated(x, w, w, residual=torch.zeros(3, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        tr.FeedForward(8, 16, activation="gelu")
    assert float(tr.clip_grad_norm([torch.nn.Parameter(torch.zeros(3))], 1.0)) == 0.0  # no gradient
    assert "hidden=16" in repr(tr.FeedForward(8, 16))


def test_w8_formula():
    """The stored weights are within half a step of the latent ones, and the
    storage holds them where the header says."""
    rng = np.random.default_rng(3)
    w = (0.02 * rng.standard_normal((17, 68))).astype(np.float32)
    w[5] = 0
    v, s = ref.w8_quant(w)
    assert np.all(np.abs(w - v * s[:, None].astype(np.float64)) <= 0.5 * s[:, None] * (1 + 1e-5))
    assert s[5] == 1 and not v[5].any()
    codes = ref.w8_pack(v).reshape(2, 2, 4, 16, 16)
    for n, k in ((0, 0), (16, 67), (3, 40), (15, 63), (7, 64)):
        assert codes[n // 16, k // 64, k % 64 // 16, n % 16, k % 16] == v[n, k]
    assert np.count_nonzero(codes) == np.count_nonzero(v)


def test_relu2_gradients_are_exact_in_fp32():
    """The kernels make dg and du of relu2 in fp32: three bf16 factors and a
    power of two have a product of at most 24 significant bits."""
    rng = np.random.default_rng(4)
    da, g, u = (oracle.bf16_to_f32(oracle.f32_to_bf16(rng.standard_normal(20000).astype(np.float32))) for _ in range(3))
    r = np.maximum(g, np.float32(0))
    dg, du = np.float32(2) * ((da * u) * r), (da * r) * r
    f = np.float64
    assert np.array_equal(dg.astype(f), 2 * da.astype(f) * u * r) and np.array_equal(du.astype(f), da.astype(f) * r * r)


# ---------------------------------------------------------------- plans

PLAN_SRC = r"""
#include "codes_plan.hpp"
#include "backward_plan.hpp"
#include <cstdio>
#include <cstdlib>

int main(int argc, char** argv) {
  for (int i = 1; i + 2 < argc; i += 3) {
    const long long m = atoll(argv[i]), n = atoll(argv[i + 1]), k = atoll(argv[i + 2]);
    for (int gated = 0; gated < 2; ++gated) {
      const bl::CodesPlan p = m > 16 ? bl::plan_codes(m, n, k, gated) : bl::CodesPlan{-1};
      const bl::CodesConfig& C = (gated ? bl::kGatedConfigs : bl::kW8Configs)[p.cfg < 0 ? 0 : p.cfg];
      const bl::RowsPlan r = bl::plan_rows(m, n, k, gated);
      printf("%d %d %d %d %d %d %d %d %d %d %d %lld\n", p.cfg, p.slabs, p.tiles_i, p.tiles_j, p.ksplit, p.kspw, C.ti, C.tj,
             C.slab, r.wk, r.seg, (long long)r.lds);
    }
    for (int want = 3; want >= 1; --want) {
      const bool dx = want != 1, dw = want != 2;
      const bl::BackwardPlan p = bl::plan_backward(m, n, k, dx, dw, true);
      printf("%d %d %d %d %d %d %d\n", p.direct, dx ? p.cfg[0] : -1, p.ksplit[0], p.kspw[0], dw ? p.cfg[1] : -1, p.ksplit[1],
             p.kspw[1]);
    }
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """shapes -> per shape (forward plans of w8 and gated, gradient plans)."""
    tmp = tmp_path_factory.mktemp("plan")
    src, exe = tmp / "plan.cpp", tmp / "plan"
    src.write_text(PLAN_SRC)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", os.path.join(ROOT, "bit_gemm_bitlinear_amd", "csrc"), str(src), "-o",
                    str(exe)], check=True)

    def run(shapes):
        out = subprocess.run([str(exe), *(str(v) for s in shapes for v in s)], capture_output=True, text=True,
                             check=True).stdout.splitlines()
        rows = [tuple(map(int, line.split())) for line in out]
        assert len(rows) == 5 * len(shapes)
        return [(rows[5 * i:5 * i + 2], rows[5 * i + 2:5 * i + 5]) for i in range(len(shapes))]

    return run


def test_plans_cover_the_products(plans):
    rng = np.random.default_rng(7)
    shapes = [(1, 1, 4), (16, 2 ** 24, 64), (2 ** 19, 2 ** 18, 4), (2 ** 19, 16, 2 ** 17), (17, 2 ** 24, 2 ** 14), (100, 100, 2 ** 17)]
    shapes += [tuple(int(2 ** (b * rng.random())) * f for b, f in ((12, 1), (14, 1), (14, 4))) for _ in range(400)]
    for (m, n, k), (forward, _) in zip(shapes, plans(shapes)):
        for gated, (cfg, slabs, ti, tj, parts, per, rows, cols, slab, wk, seg, lds) in enumerate(forward):
            tile, mats = (256, 2) if gated else (64, 1)
            # rows kernel: the staged tokens and the sums fit, every tile has a wave
            blocks, ktiles = -(-n // 16), -(-k // tile)
            assert wk in (1, 2, 4, 8, 16) and 1 <= seg <= ktiles and lds <= 80000 and lds >= 16 * mats * 1024
            assert lds >= min(m, 16) * (-(-seg * tile // 256) * 256 + 16)
            assert -(-blocks // (16 // wk)) * 1024 < 2 ** 32 and (cfg >= 0 or -(-m // 16) <= 65535)
            if cfg < 0:
                continue
            assert m > 16 and slabs == -(-k // slab) and ti == -(-m // rows) and tj == -(-n // cols)
            assert 1 <= parts <= 16 and (parts - 1) * per < slabs <= parts * per  # no part is empty
            assert (ti * tj * parts + 7) * (512 if not gated and cols == 256 else 256) < 2 ** 32


def test_gradient_plans_cover_the_products(plans):
    rng = np.random.default_rng(8)
    shapes = [(1, 1, 4), (2048, 6912, 2560), (4096, 14336, 4096)]
    shapes += [tuple(int(2 ** (b * rng.random())) * f for b, f in ((12, 1), (13, 1), (12, 4))) for _ in range(300)]
    for (m, n, k), (_, gradients) in zip(shapes, plans(shapes)):
        for direct, c0, p0, s0, c1, p1, s1 in gradients:
            assert not direct and (c0 == 2) == (c1 == 2) or c0 < 0 or c1 < 0
            for c, parts, per, slabs in ((c0, p0, s0, 2 * -(-n // 64)), (c1, p1, s1, -(-m // 64))):
                if c >= 0:
                    assert (parts - 1) * per < slabs <= parts * per


def test_gpu_shapes_take_every_plan(plans):
    """The GPU tests' shapes by plan: every kernel and tile, whole and in parts."""
    from test_ffn_gpu import BACK, SHAPES, W8_SHAPES

    for gated, shapes in enumerate((W8_SHAPES, SHAPES)):
        seen = {(p[gated][0], p[gated][4] > 1, s[2] % 16 > 0) for s, (p, _) in zip(shapes, plans(shapes)) if s[0] > 16}
        want = {(c, p, odd) for c in range(3 if gated else 4) for p in (False, True) for odd in (False, True)}
        want = want - {(3, True, False)} | {(-1, False, False), (-1, False, True)}
        assert want <= seen, (gated, want - seen)
    tiles = set()
    for _, gradients in plans(BACK):
        _, c0, p0, _, c1, p1, _ = gradients[0]
        tiles |= {("dx", c0, p0 > 1), ("dw", c1, p1 > 1)}
    assert tiles >= {(w, c, p) for w in ("dx", "dw") for c in range(3) for p in (False, True)} - {("dw", 2, True)}


WORD_ROWS_SRC = r"""
#include "codes_plan.hpp"
#include <cstdio>
#include <cstdlib>

// Per shape and product the tile that loads words, and how many of its rows begin elsewhere
// than the product's row (or the last one, for those past it).
int main(int argc, char** argv) {
  for (int i = 1; i + 2 < argc; i += 3) {
    const long long m = atoll(argv[i]), n = atoll(argv[i + 1]), k = atoll(argv[i + 2]);
    for (int gated = 0; gated < 2; ++gated) {
      const bl::CodesPlan p = bl::plan_codes(m, n, k, gated);
      if (p.cfg < 0 || p.cfg >= bl::kCodesWordTiles || k % 16 == 0) {
        printf("-1 0\n");
        continue;
      }
      const int ti = (gated ? bl::kGatedConfigs : bl::kW8Configs)[p.cfg].ti;
      long long wrong = 0;
      for (long long i0 = 0; i0 < m; i0 += ti) {
        const uint32_t end = bl::tile_last_row(ti, (int32_t)(m - i0), (int32_t)k);
        for (int r = 0; r < ti; ++r)
          wrong += std::min((uint32_t)r * (uint32_t)k, end) != std::min<long long>(r, m - 1 - i0) * k;
      }
      printf("%d %lld\n", p.cfg, wrong);
    }
  }
  return 0;
}
"""

# Odd widths and more than 2^32 bytes of codes: (tokens, outputs, width).
WORD_ROWS = [(65552, 64, 65540), (65600, 64, 65540), (131072, 64, 32772), (524288, 16, 131068), (76411, 61, 64684)]


def test_rows_of_tiles_that_load_words(tmp_path):
    """Where each row of a tile begins, with more than 2^32 bytes of codes after it."""
    src, exe = tmp_path / "rows.cpp", tmp_path / "rows"
    src.write_text(WORD_ROWS_SRC)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", os.path.join(ROOT, "bit_gemm_bitlinear_amd", "csrc"), str(src), "-o",
                    str(exe)], check=True)
    shapes = WORD_ROWS + [(33, 40, 20), (300, 19, 2 ** 17 - 4), (1705, 33, 12604), (401, 5316, 356)]
    out = subprocess.run([str(exe), *(str(v) for s in shapes for v in s)], capture_output=True, text=True,
                         check=True).stdout.splitlines()
    rows = [tuple(map(int, line.split())) for line in out]
    assert len(rows) == 2 * len(shapes)
    # the GPU test's shape takes such a tile in both products
    assert rows[0][0] in (0, 1) and rows[1][0] in (0, 1)
    for i, shape in enumerate(shapes):
        assert rows[2 * i][1] == 0 and rows[2 * i + 1][1] == 0, (shape, rows[2 * i:2 * i + 2])
