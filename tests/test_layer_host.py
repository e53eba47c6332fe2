"""Host-side checks of the operators around the product (bitlinear_layer.h)
that need no GPU: exports, refusals (every call below fails validation, so no
kernel is launched), the oracle's formulas against differences, and the 4-bit
storage against its description."""

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import oracle
from oracle import layer as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, ESHAPE, EALIGN, EWORKSPACE = 0, 1, 2, 3, 4
P = ctypes.c_void_p
A = [P(0x1000000000 * (i + 1)) for i in range(12)]  # aligned, far apart, never dereferenced
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
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "bitlinear_layer.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(bitlinear_\w+)\s*\(", text)))
    assert len(names) == 12
    out = subprocess.run(["nm", "-D", "--defined-only", bl.LIB_PATH], capture_output=True, text=True).stdout
    assert set(names) <= set(re.findall(r"\bT (bitlinear_\w+)", out))
    assert set(names) <= set(bl._SIGS)


BAD_SHAPES = [(0, 64), (-1, 64), (1, 0), (1, 66), (1, 2 ** 22 + 4), (2 ** 24 + 1, 64)]


def norm(lib, m=2, k=64, x=A[0], res=A[1], w=A[2], wt=1, eps=1e-5, h=A[3], rstd=A[4], n=None, q=A[5], xs=A[6]):
    return lib.bitlinear_rms_norm_quant(m, k, x, res, w, wt, eps, h, rstd, n, q, xs, None)


def test_norm_refusals(lib):
    for m, k in BAD_SHAPES:
        assert norm(lib, m, k) == ESHAPE
    assert norm(lib, x=None) == EINVAL
    for bad in (dict(w=None), dict(wt=0), dict(wt=3), dict(wt=-1)):
        assert norm(lib, **bad) == EINVAL
    for eps in (0.0, -1e-5, 1e-61, 1e61, float("nan"), float("inf")):
        assert norm(lib, eps=eps) == EINVAL
    assert norm(lib, q=None) == EINVAL and norm(lib, xs=None) == EINVAL
    assert norm(lib, h=None, rstd=None, q=None, xs=None) == EINVAL  # nothing to write
    for name in ("x", "res", "w", "h", "rstd", "n", "q", "xs"):
        assert norm(lib, **{name: ODD}) == EALIGN, name
    # overlaps: h may be x or the residual exactly, nothing else
    shifted = P(A[0].value + 64)
    for bad in (dict(h=shifted), dict(n=A[0]), dict(q=A[0]), dict(q=A[1]), dict(rstd=A[2]), dict(h=A[2]),
                dict(q=A[3]), dict(xs=A[4]), dict(n=A[5])):
        assert norm(lib, **bad) == EINVAL, bad


def nback(lib, m=20, k=64, dn=A[0], h=A[1], rstd=A[2], w=A[3], wt=2, dh=A[4], dx=A[5], dw=A[6], acc=0, ws=A[7], n=BIG):
    return lib.bitlinear_rms_norm_quant_backward(m, k, dn, h, rstd, w, wt, dh, dx, dw, acc, ws, n, None)


def test_norm_backward_refusals(lib):
    need = lib.bitlinear_rms_norm_quant_backward_workspace_bytes
    for m, k in BAD_SHAPES:
        assert nback(lib, m, k) == ESHAPE
        assert need(m, k, 1) == 0
    for name in ("dn", "h", "rstd", "dx"):
        assert nback(lib, **{name: None}) == EINVAL
    for bad in (dict(w=None), dict(wt=0), dict(wt=7), dict(acc=2), dict(acc=-1)):
        assert nback(lib, **bad) == EINVAL
    for name in ("dn", "h", "rstd", "w", "dh", "dx", "dw", "ws"):
        assert nback(lib, **{name: ODD}) == EALIGN, name
    size = need(20, 64, 1)
    assert size >= 64 * 4 and need(20, 64, 0) == 0 and need(8, 64, 1) == 0
    assert nback(lib, ws=None) == EWORKSPACE and nback(lib, n=ctypes.c_size_t(size - 1)) == EWORKSPACE
    for bad in (dict(dx=A[1]), dict(dx=P(A[0].value + 64)), dict(dw=A[0]), dict(dw=A[3]), dict(ws=A[1]), dict(ws=A[5]),
                dict(ws=A[6])):
        assert nback(lib, **bad) == EINVAL, bad


def test_restore_refusals(lib):
    f = lib.bitlinear_restore_activations
    for m, k in BAD_SHAPES:
        assert f(m, k, A[0], A[1], A[2], None) == ESHAPE
    for i in range(3):
        args = [A[0], A[1], A[2]]
        args[i] = None
        assert f(2, 64, *args, None) == EINVAL
        args[i] = ODD
        assert f(2, 64, *args, None) == EALIGN
    assert f(2, 64, A[0], A[1], A[0], None) == EINVAL


def back(lib, m=512, n=2048, k=2048, dy=A[0], packed=A[1], layout=0, s=A[2], res=None, dx=A[3], q=A[4], xs=A[5],
         dw=A[6], db=A[7], acc=0, ws=A[8], size=BIG):
    return lib.bitlinear_backward(m, n, k, dy, packed, layout, s, res, dx, q, xs, dw, db, acc, ws, size, None)


def test_backward_refusals(lib):
    need = lib.bitlinear_backward_workspace_bytes
    for m, n, k in [(0, 32, 256), (4, 0, 256), (4, 32, 0), (4, 32, 6), (2 ** 21 + 1, 4, 4), (4, 2 ** 21 + 1, 4),
                    (4, 4, 2 ** 22 + 4), (2 ** 21, 2 ** 21, 4), (2 ** 21, 4, 2 ** 20), (4, 2 ** 21, 2 ** 20)]:
        assert back(lib, m, n, k) == ESHAPE, (m, n, k)
        assert need(m, n, k, 1, 1) == 0
    assert need(512, 2048, 2048, 0, 0) == 0
    assert need(512, 2048, 2048, 1, 1) > max(need(512, 2048, 2048, 1, 0), need(512, 2048, 2048, 0, 1)) > 0
    for bad in (dict(dy=None), dict(packed=None), dict(s=None), dict(q=None), dict(xs=None), dict(layout=2),
                dict(layout=-1), dict(acc=2), dict(dx=None, dw=None, db=None), dict(dw=None), dict(dx=None, res=A[9])):
        assert back(lib, **bad) == EINVAL, bad
    assert back(lib, n=33, layout=1) == ESHAPE and back(lib, k=260, layout=1) == ESHAPE
    for name in ("dy", "packed", "s", "res", "dx", "q", "xs", "dw", "db", "ws"):
        assert back(lib, **{name: ODD}) == EALIGN, name
    size = need(512, 2048, 2048, 1, 1)
    assert back(lib, ws=None) == EWORKSPACE and back(lib, size=ctypes.c_size_t(size - 1)) == EWORKSPACE
    for bad in (dict(dx=A[0]), dict(dw=A[4]), dict(db=A[6]), dict(ws=A[3]), dict(ws=A[0]), dict(res=P(A[3].value + 64)),
                dict(res=A[6]), dict(res=A[8])):
        assert back(lib, **bad) == EINVAL, bad


def test_backward_workspace_holds_every_plan(lib):
    """Sizes over the range: none (the one-launch kernel), or the operands'
    slabs and no more than sixteen parts of the outputs besides."""
    need = lib.bitlinear_backward_workspace_bytes
    rng = np.random.default_rng(1)
    sizes = set()
    for _ in range(2000):
        m, n, k = (int(2 ** rng.uniform(0, 14)) for _ in range(3))
        k = 4 * max(1, k // 4)
        mp, np_ = -(-m // 64) * 64, -(-n // 64) * 64
        least = (2 * np_ * m if n % 64 else 0) + np_ * k // 4 + 2 * mp * (n + k)
        size = need(m, n, k, 1, 1)
        assert size == 0 or least <= size <= least + 4 * mp // 64 * n + 64 * k * (m + n) + 8 * 256
        sizes.add(size > 0)
    assert sizes == {False, True}


def w4(lib, m=3, n=20, k=256, group=64, q=A[0], xs=A[1], codes=A[2], scales=A[3], bias=None, y=A[4]):
    return lib.bitlinear_w4_forward(m, n, k, group, q, xs, codes, scales, bias, y, None)


def test_w4_refusals(lib):
    for m, n, k in [(0, 20, 256), (3, 0, 256), (3, 20, 0), (3, 20, 258), (2 ** 19 + 1, 1, 64), (1, 2 ** 24 + 1, 64)]:
        assert w4(lib, m, n, k) == ESHAPE, (m, n, k)
    for group in (0, 16, 48, 2048, -64):
        assert w4(lib, group=group) == EINVAL
        assert lib.bitlinear_w4_scales_bytes(20, 256, group) == 0
    assert w4(lib, k=256 + 32, group=64) == ESHAPE
    for name in ("q", "xs", "codes", "scales", "y"):
        assert w4(lib, **{name: None}) == EINVAL
        assert w4(lib, **{name: ODD}) == EALIGN
    assert w4(lib, bias=ODD) == EALIGN
    for bad in (dict(y=A[0]), dict(y=A[2]), dict(bias=A[4])):
        assert w4(lib, **bad) == EINVAL
    assert lib.bitlinear_w4_codes_bytes(20, 160) == 2 * 2 * 1024
    assert lib.bitlinear_w4_scales_bytes(20, 160, 32) == 2 * 5 * 32
    for f, args in ((lib.bitlinear_w4_pack, (A[0], 20, 256, 64, A[1], A[2])),):
        for i in (0, 4, 5):
            bad = list(args)
            bad[i] = None
            assert f(*bad, None) == EINVAL
        assert f(A[0], 20, 256, 64, A[0], A[2], None) == EINVAL
    assert lib.bitlinear_w4_unpack(A[0], A[1], 20, 256, 64, A[0], None) == EINVAL
    assert lib.bitlinear_w4_unpack(A[0], A[1], 20, 250, 64, A[2], None) == ESHAPE


def test_forward_quantized_refusals(bl, lib):
    def call(x=0, q=0x2000000000, xs=0x3000000000, codes=True, **kw):
        p = (bl.Projection * 1)(bl.Projection(x, A[0].value, A[1].value, A[2].value, 16, 64))
        c = (bl.Codes * 1)(bl.Codes(q, xs))
        return lib.bitlinear_forward_grouped_quantized(kw.get("count", 1), p, c if codes else None, kw.get("m", 2),
                                                       A[3], kw.get("size", BIG), None)

    assert call(x=0x5000000000) == EINVAL  # bf16 activations as well
    assert call(q=0) == EINVAL and call(xs=0) == EINVAL and call(codes=False) == EINVAL
    assert call(q=0x2000000008) == EALIGN and call(xs=0x3000000004) == EALIGN
    assert call(count=0) == EINVAL and call(count=17) == EINVAL and call(m=0) == ESHAPE
    assert call(size=ctypes.c_size_t(16)) == EWORKSPACE


def test_binding_refuses_host_tensors(bl):
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(2, 64, dtype=torch.int8), torch.ones(2)
    for call in (lambda: bl.rms_norm_quant(x), lambda: bl.restore_activations(q, s),
                 lambda: bl.rms_norm_quant_backward(x, x, s), lambda: bl.BackwardCall(x, q, s),
                 lambda: bl.backward_input(x, torch.zeros(64, 16, dtype=torch.uint8), s),
                 lambda: bl.pack_weights_w4(torch.zeros(4, 64)), lambda: bl.forward_quantized(q, s, q, s),
                 lambda: bl.forward_w4(q, s, bl.W4Weights(q, x, 4, 64, 32))):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        bl.unpack_weights_w4(bl.W4Weights(q, x, 4, 64, 0))
    with pytest.raises(ValueError):
        bl.unpack_weights_w4(bl.W4Weights(q, x, 0, 64, 32))


# ------------------------------------------------------------------ formulas

@pytest.mark.parametrize("weight", [False, True])
def test_norm_gradient_formula_against_differences(weight):
    rng = np.random.default_rng(1)
    m, k, eps = 4, 24, 1e-3
    h, dn, dh = (rng.standard_normal((m, k)) for _ in range(3))
    h[2] = 0  # a padded row
    w = 1 + rng.standard_normal(k) if weight else None
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    out = ref.rms_norm_quant_backward(dn, h, rstd, w, dh)

    def loss(hh, ww):
        return (ref.norm_value(hh, ww, eps) * dn).sum() + (hh * dh).sum()

    t = 1e-6
    for i in range(m):
        for j in range(0, k, 5):
            a, b = h.copy(), h.copy()
            a[i, j] += t
            b[i, j] -= t
            assert abs((loss(a, w) - loss(b, w)) / (2 * t) - out["dx"][i, j]) <= 1e-6 * (1 + abs(out["dx"][i, j]))
    if weight:
        for j in range(k):
            a, b = w.copy(), w.copy()
            a[j] += t
            b[j] -= t
            assert abs((loss(h, a) - loss(h, b)) / (2 * t) - out["dweight"][j]) <= 1e-6 * (1 + abs(out["dweight"][j]))


def test_w4_storage_description():
    """The header's byte formula, every weight in a place of its own."""
    for n, k in ((16, 128), (33, 160), (5, 384)):
        kt = -(-k // 128)
        places = [ref.w4_position(i, j, kt) for i in range(n) for j in range(k)]
        assert len(set(places)) == n * k
        nb = -(-n // 16)
        for (i, j), (off, sh) in zip(((i, j) for i in range(n) for j in range(k)), places):
            at = np.ravel_multi_index((i // 16, j // 128, (j % 32) // 8, i % 16, 4 * ((j % 128) // 32) + j % 4),
                                      (nb, kt, 4, 16, 16))
            assert off == at and sh == (4 if j % 8 < 4 else 0)


def test_oracle_norm_matches_the_activation_quantization():
    rng = np.random.default_rng(2)
    x = oracle.f32_to_bf16(rng.standard_normal((3, 40)).astype(np.float32))
    r = oracle.f32_to_bf16(rng.standard_normal((3, 40)).astype(np.float32))
    q, s, h, rstd, n = ref.rms_norm_quant(x, r, None, 1e-5)
    assert np.array_equal(h, oracle.add_bf16(x, r))
    q2, s2 = oracle.act_quant(n)
    assert np.array_equal(q, q2) and np.array_equal(s, s2)
    # unit root mean square, to the rounding to bf16 and eps
    assert np.all(np.abs((oracle.bf16_to_f32(n).astype(np.float64) ** 2).mean(1) - 1) <= 2 ** -6)


# ------------------------------------------------------------------ training form

def test_training_refuses_weights_of_another_width(bl):
    """Before anything else, so host tensors show it."""
    from bit_gemm_bitlinear_amd import training as tr

    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    for shape in ((16, 4096), (16, 1024), (16, 64), (16, 252), (256,), (2, 16, 256)):
        w = torch.zeros(shape)
        for call in (lambda: tr.linear(x, w), lambda: tr.norm_linear(x, [w]), lambda: tr.norm_linear(x, [w], None, x),
                     lambda: tr.norm_linear(x, [torch.zeros(16, 256), w])):
            with pytest.raises(ValueError, match="weight"):
                call()


def test_forward_quantized_refuses_overlaps(bl, lib):
    """Outputs and workspace apart from what the call reads and from each
    other; a projection's residual may be its own output, exactly."""
    size = ctypes.c_size_t(1 << 20)
    names = ("q", "xs", "packed", "ws", "bias", "res", "y")

    def call(m=20, wsp=A[10].value, **kw):
        p, c = (bl.Projection * 2)(), (bl.Codes * 2)()
        for i in range(2):
            at = {n: 0x1000000000 * (1 + len(names) * i + j) + (1 << 45) for j, n in enumerate(names)}
            at.update({n[:-1]: v for n, v in kw.items() if n[-1] == str(i)})
            p[i] = bl.Projection(0, at["packed"], at["ws"], at["y"], 48, 64, 0, 0, at["bias"], at["res"])
            c[i] = bl.Codes(at["q"], at["xs"])
        return lib.bitlinear_forward_grouped_quantized(2, p, c, m, P(wsp), size, None)

    y = 1 << 44
    sizes = dict(q=20 * 64, xs=80, packed=48 * 16, ws=4, bias=96, res=20 * 96)
    for name, n in sizes.items():
        for i in (0, 1):
            last = y + (20 * 96 - 1) // 16 * 16  # the output's last 16 bytes
            for start in (y + 16, last, y - (n - 1) // 16 * 16):
                assert call(**{"y0": y, f"{name}{i}": start}) == EINVAL, (name, i, start - y)
    assert call(y0=y, y1=y) == EINVAL and call(y0=y, y1=y + 20 * 96 - 16) == EINVAL
    assert call(y0=y, res1=y) == EINVAL  # another projection's output
    for name in ("q", "xs", "packed", "ws", "bias", "res", "y"):
        assert call(wsp=y, **{f"{name}1": y + 64}) == EINVAL, name
    assert call(wsp=0, y0=y, q0=y) == EWORKSPACE  # checked before


# ------------------------------------------------------------------ the device of a call

class _OnDevice(torch.Tensor):
    """A host tensor that says it is on cuda:1."""
    device = property(lambda self: torch.device("cuda", 1))
    is_cuda = property(lambda self: True)


def test_calls_make_their_tensors_device_current(bl, monkeypatch):
    """Every call of the binding enqueues on the current stream of its tensors'
    device with that device current, whichever is current around it: the
    library launches on the current one."""
    class Device:
        def __init__(self, device):
            self.index = torch.device(device).index if not isinstance(device, int) else device

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *exc):
            current.pop()

    current, calls = [0], []
    real = {n: getattr(bl._lib, n) for n in bl._SIGS}

    class Lib:
        def __getattr__(self, name):
            if "bytes" in name or "launches" in name or "status" in name:
                return real[name]

            def entry(*args):
                stream = args[-1]
                calls.append((name, current[-1], stream.value if isinstance(stream, P) else stream))
                return OK
            return entry

    def on_device(make):
        return lambda *a, **kw: make(*a, **{k: v for k, v in kw.items() if k != "device"}).as_subclass(_OnDevice)

    class Stream:
        def __init__(self, index):
            self.cuda_stream = 100 + index

    monkeypatch.setattr(bl, "_lib", Lib())
    monkeypatch.setattr(bl, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream(torch.device(d).index))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch, "empty", on_device(torch.empty))
    monkeypatch.setattr(torch, "zeros", on_device(torch.zeros))
    m, n, k = 3, 16, 256
    x, y = torch.zeros(m, k, dtype=torch.bfloat16), torch.zeros(m, n, dtype=torch.bfloat16)
    w, packed, s = torch.zeros(n, k), torch.zeros(n, k // 4, dtype=torch.uint8), torch.zeros(4)
    q, xs, tiled = torch.zeros(m, k, dtype=torch.int8), torch.zeros(m), torch.zeros(1, 4 * k, dtype=torch.uint8)
    bias = torch.zeros(n, dtype=torch.bfloat16)
    made = [
        lambda: bl.pack_weights(w), lambda: bl.unpack_weights(packed), lambda: bl.export_bf16(packed, s),
        lambda: bl.forward_latent(x, w), lambda: bl.tile_weights(packed), lambda: bl.untile_weights(tiled),
        lambda: bl.act_quant(x), lambda: bl.forward(x, packed, s), lambda: bl.forward(x, tiled, s),
        lambda: bl.forward(x, packed, s, bias=bias), lambda: bl.forward_grouped([x, x], [packed, tiled], [s, s]),
        lambda: bl.forward_grouped_inspect([x], [packed], [s]), lambda: bl.forward_acc(q, packed),
        lambda: bl.forward_acc(q, tiled), lambda: bl.rms_norm_quant(x), lambda: bl.rms_norm_quant_backward(x, x, xs),
        lambda: bl.restore_activations(q, xs), lambda: bl.forward_quantized(q, xs, packed, s),
        lambda: bl.backward_input(y, packed, s), lambda: bl.backward_weight(y, q, xs),
        lambda: bl.unpack_weights_w4(bl.pack_weights_w4(w)), lambda: bl.forward_w4(q, xs, bl.pack_weights_w4(w)),
    ]
    for around in (0, 1):
        current[:] = [around]
        for make in made:
            calls.clear()
            make()
            assert calls and all(c[1:] == (1, 101) for c in calls), calls
            assert current == [around]
    for stream, want in ((7, 7), (0, 0)):
        calls.clear()
        bl.GroupedCall([x], [packed], [s])(stream)
        assert calls[0][1] == 1 and (calls[0][2] or 0) == want


# ------------------------------------------------------------------ plan of the gradients

BACKWARD_PLAN_SRC = r'''
#include "backward_plan.hpp"
#include <cstdio>
#include <cstdlib>

int main(int argc, char** argv) {
  for (int i = 1; i + 2 < argc; i += 3)
    for (int want = 3; want >= 1; --want) {  // both, dx, dw
      const bool dx = want != 1, dw = want != 2;
      const bl::BackwardPlan p = bl::plan_backward(atoll(argv[i]), atoll(argv[i + 1]), atoll(argv[i + 2]), dx, dw);
      if (p.direct)
        printf("one\n");
      else
        printf("%d %d %d %d %d %d\n", dx ? bl::kConfigs[p.cfg[0]].ti : 0, p.ksplit[0], p.kspw[0],
               dw ? bl::kConfigs[p.cfg[1]].ti : 0, p.ksplit[1], p.kspw[1]);
    }
  return 0;
}
'''


def backward_plans(tmp_path, shapes):
    """{shape: plans of both gradients, dx alone, dw alone}: "one" or (tile of
    dx, parts, slabs a part, tile of dw, parts, slabs a part; tile 0: not wanted)."""
    src, exe = tmp_path / "backward_plan.cpp", tmp_path / "backward_plan"
    src.write_text(BACKWARD_PLAN_SRC)
    csrc = os.path.join(ROOT, "bit_gemm_bitlinear_amd", "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe), *(str(v) for s in shapes for v in s)], capture_output=True, text=True,
                         check=True).stdout.splitlines()
    plans = ["one" if line == "one" else tuple(map(int, line.split())) for line in out]
    assert len(plans) == 3 * len(shapes)
    return {s: plans[3 * i:3 * i + 3] for i, s in enumerate(shapes)}


def test_gradient_shapes_take_the_plans_they_are_for(tmp_path):
    """The GPU tests' shapes by plan, every tile size and split among them."""
    from test_layer_gpu import BY_PLAN, PLANS

    tiles, parts = set(), set()
    for shape, plans in backward_plans(tmp_path, list(BY_PLAN)).items():
        for plan, want in zip(plans, BY_PLAN[shape]):
            if plan == "one" or want == "one":
                assert plan == want, (shape, plan)
                continue
            tx, px, _, tw, pw, _ = plan
            assert want == (tx or None, px if tx else None, tw or None, pw if tw else None), (shape, plan)
            for product, tile, p in (("dx", tx, px), ("dw", tw, pw)):
                if tile:
                    tiles.add((product, tile, p > 1, all(shape[i] % 64 for i in range(3))))
    # either product on every tile size, whole and in parts, at ragged sizes
    for product in ("dx", "dw"):
        for tile in (64, 128, 256):
            for split in (False, True):
                assert (product, tile, split, True) in tiles, (product, tile, split)
    got = [p[0] for p in backward_plans(tmp_path, PLANS).values()]
    assert got[0] == "one"
    assert [(p[0], p[1] > 1, p[3], p[4] > 1) for p in got[1:]] == [
        (64, False, 64, False), (64, True, 64, False), (64, False, 64, True), (128, False, 128, False),
        (256, True, 256, False)]


def test_gradient_plans_cover_their_sums(tmp_path):
    """Every split covers its sum with no empty part and at most 16 parts, and
    the library's workspace queries follow the same plan."""
    from bit_gemm_bitlinear_amd import bitlinear

    need = bitlinear.lib().bitlinear_backward_workspace_bytes
    rng = np.random.default_rng(4)
    shapes = []
    for _ in range(300):
        m, n, k = (int(2 ** rng.uniform(0, 14)) for _ in range(3))
        shapes.append((m, n, 4 * max(1, k // 4)))
    for (m, n, k), plans in backward_plans(tmp_path, sorted(set(shapes))).items():
        for plan, dx, dw in zip(plans, (1, 1, 0), (1, 0, 1)):
            assert (need(m, n, k, dx, dw) == 0) == (plan == "one")
            if plan == "one":
                continue
            for want, c, parts, each in ((dx, n, *plan[1:3]), (dw, m, *plan[4:6])):
                slabs = -(-c // 64)
                if want:
                    assert 1 <= parts <= 16 and parts * each >= slabs > (parts - 1) * each, (m, n, k, plan)
