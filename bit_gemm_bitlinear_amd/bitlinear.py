"""ctypes binding over libbitlinear.so (C ABI in include/bitlinear.h,
include/bitlinear_layer.h and include/bitlinear_ffn.h).

Argument marshalling only: every step of the BitLinear forward pass runs in
the library's HIP kernels.  PyTorch provides device memory and the current
HIP stream.  Importing this module loads the library and raises ImportError
if it has not been built (``python -m bit_gemm_bitlinear_amd.build``); there
is no fallback implementation.
"""

from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Sequence

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libbitlinear.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m bit_gemm_bitlinear_amd.build` "
        "(hipcc for gfx950); the BitLinear kernels have no fallback")

_lib = ctypes.CDLL(LIB_PATH)

_i64, _i32, _sz, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p
_dbl, _flt = ctypes.c_double, ctypes.c_float


class Projection(ctypes.Structure):
    """bl_projection: one projection of a grouped forward call."""
    _fields_ = [("x", _vp), ("packed", _vp), ("w_scale", _vp), ("y", _vp),
                ("n", _i64), ("k", _i64), ("layout", _i32), ("reserved", _i32),
                ("bias", _vp), ("residual", _vp)]


class Inspect(ctypes.Structure):
    """bl_inspect: side outputs of a forward call (codes, scales, code sums,
    int32 accumulators)."""
    _fields_ = [("q", _vp), ("x_scale", _vp), ("qsum", _vp), ("acc", _vp)]


class Codes(ctypes.Structure):
    """bl_codes: int8 activations of a projection (codes and scales)."""
    _fields_ = [("q", _vp), ("x_scale", _vp)]


class Gradient(ctypes.Structure):
    """bl_gradient: one tensor of a gradient norm or clipping call."""
    _fields_ = [("g", _vp), ("out", _vp), ("numel", _i64), ("type", _i32), ("reserved", _i32)]


LAYOUT_ROWS = 0   # BL_LAYOUT_ROWS: packed uint8 [N, K/4]
LAYOUT_TILED = 1  # BL_LAYOUT_TILED: uint8 [N/16, 4*K], one row per block of 16 weight rows


_SIGS = {
    "bitlinear_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "bitlinear_abi_version": (ctypes.c_int, []),
    "bitlinear_pack_workspace_bytes": (_sz, [_i64, _i64]),
    "bitlinear_pack_weights": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp, _sz, _vp]),
    "bitlinear_unpack_weights": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp]),
    "bitlinear_export_bf16": (ctypes.c_int, [_vp, _i64, _i64, _i32, _vp, _vp, _vp]),
    "bitlinear_forward_latent_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "bitlinear_forward_latent": (ctypes.c_int, [_i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _sz,
                                                _vp]),
    "bitlinear_tile_weights": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp]),
    "bitlinear_untile_weights": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp]),
    "bitlinear_act_quant": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "bitlinear_forward_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "bitlinear_forward": (ctypes.c_int, [_i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "bitlinear_forward_tiled": (ctypes.c_int, [_i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _sz,
                                               _vp]),
    "bitlinear_forward_grouped_workspace_bytes": (_sz, [_i32, ctypes.POINTER(Projection), _i64]),
    "bitlinear_forward_grouped_launches": (_i32, [_i32, ctypes.POINTER(Projection), _i64]),
    "bitlinear_forward_grouped": (ctypes.c_int, [_i32, ctypes.POINTER(Projection), _i64, _vp,
                                                 _sz, _vp]),
    "bitlinear_forward_grouped_inspect": (ctypes.c_int, [_i32, ctypes.POINTER(Projection), _i64,
                                                         ctypes.POINTER(Inspect), _vp, _i32, _vp,
                                                         _sz, _vp]),
    "bitlinear_forward_grouped_noalloc": (ctypes.c_int, [_i32, ctypes.POINTER(Projection), _i64,
                                                         _vp]),
    "bitlinear_forward_acc": (ctypes.c_int, [_i64, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "bitlinear_forward_acc_tiled": (ctypes.c_int, [_i64, _i64, _i64, _vp, _vp, _vp, _vp, _sz,
                                                   _vp]),
    # include/bitlinear_layer.h
    "bitlinear_rms_norm_quant": (ctypes.c_int, [_i64, _i64, _vp, _vp, _vp, _i32, _dbl, _vp, _vp,
                                                _vp, _vp, _vp, _vp]),
    "bitlinear_rms_norm_quant_backward_workspace_bytes": (_sz, [_i64, _i64, _i32]),
    "bitlinear_rms_norm_quant_backward": (ctypes.c_int, [_i64, _i64, _vp, _vp, _vp, _vp, _i32, _vp,
                                                         _vp, _vp, _i32, _vp, _sz, _vp]),
    "bitlinear_restore_activations": (ctypes.c_int, [_i64, _i64, _vp, _vp, _vp, _vp]),
    "bitlinear_forward_grouped_quantized": (ctypes.c_int, [_i32, ctypes.POINTER(Projection),
                                                           ctypes.POINTER(Codes), _i64, _vp, _sz,
                                                           _vp]),
    "bitlinear_backward_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32, _i32]),
    "bitlinear_backward": (ctypes.c_int, [_i64, _i64, _i64, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp,
                                          _vp, _vp, _i32, _vp, _sz, _vp]),
    "bitlinear_w4_codes_bytes": (_sz, [_i64, _i64]),
    "bitlinear_w4_scales_bytes": (_sz, [_i64, _i64, _i64]),
    "bitlinear_w4_pack": (ctypes.c_int, [_vp, _i64, _i64, _i64, _vp, _vp, _vp]),
    "bitlinear_w4_unpack": (ctypes.c_int, [_vp, _vp, _i64, _i64, _i64, _vp, _vp]),
    "bitlinear_w4_forward": (ctypes.c_int, [_i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                            _vp]),
    # include/bitlinear_ffn.h
    "bitlinear_gated_weights_bytes": (_sz, [_i64, _i64]),
    "bitlinear_gated_weights": (ctypes.c_int, [_i64, _i64, _vp, _i32, _vp, _i32, _vp, _vp]),
    "bitlinear_gated_forward_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "bitlinear_gated_forward": (ctypes.c_int, [_i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i32, _vp,
                                               _vp, _vp, _vp, _sz, _vp]),
    "bitlinear_gated_backward_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32, _i32]),
    "bitlinear_gated_backward": (ctypes.c_int, [_i64, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _i32, _vp,
                                                _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp,
                                                _sz, _vp]),
    "bitlinear_w8_codes_bytes": (_sz, [_i64, _i64]),
    "bitlinear_w8_pack": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "bitlinear_w8_unpack": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp]),
    "bitlinear_w8_forward_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "bitlinear_w8_forward": (ctypes.c_int, [_i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                            _vp]),
    "bitlinear_grad_norm_workspace_bytes": (_sz, [_i32, ctypes.POINTER(Gradient)]),
    "bitlinear_grad_norm": (ctypes.c_int, [_i32, ctypes.POINTER(Gradient), _vp, _vp, _sz, _vp]),
    "bitlinear_clip_gradients": (ctypes.c_int, [_i32, ctypes.POINTER(Gradient), _flt, _vp, _vp, _sz,
                                                _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

STATUS = {0: "BL_OK", 1: "BL_EINVAL", 2: "BL_ESHAPE", 3: "BL_EALIGN", 4: "BL_EWORKSPACE",
          5: "BL_EHIP"}


class BitLinearError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        msg = _lib.bitlinear_status_string(status).decode()
        super().__init__(f"{STATUS.get(status, status)}: {msg}")


def lib() -> ctypes.CDLL:
    return _lib


# The current stream's handle of a device index, and the current device: what
# torch.cuda.current_stream and current_device look up, without the objects
# around it (1.9 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(fn, args, device: torch.device, stream=None) -> None:
    """Calls an entry point on `device`'s current stream (or the given one),
    with that device current: a kernel goes to the current device."""
    if torch.cuda.current_device() == device.index:
        status = fn(*args, _raw_stream(device.index) if stream is None else stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(device.index) if stream is None else stream)
    if status:
        raise BitLinearError(status)


def _ptr(t: torch.Tensor):
    return ctypes.c_void_p(t.data_ptr())


def _require(t: torch.Tensor, dtype, ndim, name, shape=None, device=None):
    """Checks a tensor handed to the library: a contiguous device tensor of
    the given dtype and rank (and shape and device, when given).  The kernels
    trust these; a host tensor or a short buffer would be read or written out
    of bounds on the GPU."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _require_scale(s: torch.Tensor, device, name="w_scale"):
    """A weight scale: fp32 device tensor with at least one element."""
    if not isinstance(s, torch.Tensor) or not s.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if s.dtype != torch.float32 or s.numel() < 1:
        raise TypeError(f"{name} must be float32 with at least one element")
    if s.device != device:
        raise ValueError(f"{name} is on {s.device}, expected {device}")


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _workspace(nbytes: int, device, workspace):
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda:
            raise TypeError("workspace must be a CUDA (HIP) tensor")
        if workspace.device != device:
            raise ValueError(f"workspace is on {workspace.device}, expected {device}")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if _nbytes(workspace) < nbytes:
            raise ValueError("workspace too small")
        return workspace
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


# --------------------------------------------------------------------------

def pack_weights(w: torch.Tensor):
    """Latent fp32 weights [N, K] -> (packed uint8 [N, K/4], w_scale fp32 [1])."""
    _require(w, torch.float32, 2, "w")
    n, k = w.shape
    packed = torch.empty((n, k // 4), dtype=torch.uint8, device=w.device)
    w_scale = torch.empty(4, dtype=torch.float32, device=w.device)[:1]
    ws = _workspace(_lib.bitlinear_pack_workspace_bytes(n, k), w.device, None)
    _launch(_lib.bitlinear_pack_weights,
            (_ptr(w), n, k, _ptr(packed), _ptr(w_scale), _ptr(ws), _nbytes(ws)), w.device)
    return packed, w_scale


def unpack_weights(packed: torch.Tensor) -> torch.Tensor:
    """Packed [N, K/4] -> int8 [N, K] values c - 1."""
    _require(packed, torch.uint8, 2, "packed")
    n, kb = packed.shape
    u = torch.empty((n, 4 * kb), dtype=torch.int8, device=packed.device)
    _launch(_lib.bitlinear_unpack_weights, (_ptr(packed), n, 4 * kb, _ptr(u)), packed.device)
    return u


def export_bf16(packed: torch.Tensor, w_scale: torch.Tensor, k: int | None = None) -> torch.Tensor:
    """The "universal" bf16 weights u / w_scale, [N, K] bf16, from packed
    weights in either layout (K is inferred for the row-major layout; give it
    for the tiled one, where [N/16, 4K] is ambiguous with row-major)."""
    _require(packed, torch.uint8, 2, "packed")
    _require_scale(w_scale, packed.device)
    if k is None:
        k = 4 * packed.shape[1]
    n, layout = weight_layout(packed, k)
    out = torch.empty((n, k), dtype=torch.bfloat16, device=packed.device)
    _launch(_lib.bitlinear_export_bf16, (_ptr(packed), n, k, layout, _ptr(w_scale), _ptr(out)),
            packed.device)
    return out


def forward_latent(x: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None):
    """The forward pass on latent fp32 weights [N, K], ternarized on the fly
    (exact absmean, then block-wise packing, then the forward).  Returns
    (y bf16 [M, N], w_scale fp32 [1])."""
    _require(x, torch.bfloat16, 2, "x")
    _require(w, torch.float32, 2, "w", device=x.device)
    m, k = x.shape
    n = w.shape[0]
    if w.shape[1] != k:
        raise ValueError("w must be [N, K] with K = x.shape[1]")
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    _require(out, torch.bfloat16, 2, "out", shape=(m, n), device=x.device)
    w_scale = torch.empty(4, dtype=torch.float32, device=x.device)[:1]
    ws = _workspace(int(_lib.bitlinear_forward_latent_workspace_bytes(m, n, k)), x.device, None)
    _launch(_lib.bitlinear_forward_latent,
            (m, n, k, _ptr(x), _ptr(w), _ptr(w_scale), _ptr(out), _ptr(ws), _nbytes(ws)), x.device)
    return out, w_scale


def tile_weights(packed: torch.Tensor) -> torch.Tensor:
    """Row-major packed [N, K/4] -> the 16-row tiled layout, as uint8
    [N/16, 4*K] (one row per block of 16 weight rows).  N % 16 == 0 and
    K % 256 == 0."""
    _require(packed, torch.uint8, 2, "packed")
    n, kb = packed.shape
    if n % 16:
        raise ValueError("the tiled layout needs N % 16 == 0")
    tiled = torch.empty((n // 16, 16 * kb), dtype=torch.uint8, device=packed.device)
    _launch(_lib.bitlinear_tile_weights, (_ptr(packed), n, 4 * kb, _ptr(tiled)), packed.device)
    return tiled


def untile_weights(tiled: torch.Tensor) -> torch.Tensor:
    """The inverse of tile_weights: [N/16, 4*K] -> row-major [N, K/4]."""
    _require(tiled, torch.uint8, 2, "tiled")
    nb, kb16 = tiled.shape
    if kb16 % 1024:
        raise ValueError("a tiled weight row holds 16 rows of K/4 bytes, K % 256 == 0")
    n, k = 16 * nb, kb16 // 4
    packed = torch.empty((n, k // 4), dtype=torch.uint8, device=tiled.device)
    _launch(_lib.bitlinear_untile_weights, (_ptr(tiled), n, k, _ptr(packed)), tiled.device)
    return packed


def weight_layout(w: torch.Tensor, k: int):
    """(N, layout) of a weight tensor used against K input features: [N, K/4]
    is row-major, [N/16, 4*K] the tiled layout."""
    if w.shape[1] * 4 == k:
        return w.shape[0], LAYOUT_ROWS
    if w.shape[1] == 4 * k and k % 256 == 0:
        return 16 * w.shape[0], LAYOUT_TILED
    raise ValueError("packed weights do not match K")


def act_quant(x: torch.Tensor):
    """bf16 activations [M, K] -> (int8 codes [M, K], fp32 scales [M])."""
    _require(x, torch.bfloat16, 2, "x")
    m, k = x.shape
    q = torch.empty((m, k), dtype=torch.int8, device=x.device)
    s = torch.empty(max(m, 4), dtype=torch.float32, device=x.device)[:m]
    _launch(_lib.bitlinear_act_quant, (_ptr(x), m, k, _ptr(q), _ptr(s)), x.device)
    return q, s


def forward_workspace_bytes(m: int, n: int, k: int) -> int:
    return int(_lib.bitlinear_forward_workspace_bytes(m, n, k))


def forward(x: torch.Tensor, packed: torch.Tensor, w_scale: torch.Tensor,
            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
            bias: torch.Tensor | None = None, residual: torch.Tensor | None = None):
    """y = BitLinear(x) as bf16 [M, N]; `packed` in either layout.  With a bf16
    bias [N] and/or a bf16 residual [M, N] (which may be `out` itself), the
    output is (y + bias) + residual, each add rounded to bf16."""
    if bias is not None or residual is not None:
        outs = None if out is None else [out]
        return GroupedCall([x], [packed], [w_scale], outs, workspace,
                           biases=[bias], residuals=[residual])()[0]
    _require(x, torch.bfloat16, 2, "x")
    _require(packed, torch.uint8, 2, "packed", device=x.device)
    _require_scale(w_scale, x.device)
    m, k = x.shape
    n, layout = weight_layout(packed, k)
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    _require(out, torch.bfloat16, 2, "out", shape=(m, n), device=x.device)
    ws = _workspace(forward_workspace_bytes(m, n, k), x.device, workspace)
    fn = _lib.bitlinear_forward_tiled if layout == LAYOUT_TILED else _lib.bitlinear_forward
    _launch(fn, (m, n, k, _ptr(x), _ptr(packed), _ptr(w_scale), _ptr(out), _ptr(ws), _nbytes(ws)),
            x.device)
    return out


def _projections(xs, packeds, w_scales, outs, biases=None, residuals=None):
    arr = (Projection * len(xs))()
    biases = biases or [None] * len(xs)
    residuals = residuals or [None] * len(xs)
    for i, (x, p, s, y, b, r) in enumerate(zip(xs, packeds, w_scales, outs, biases, residuals)):
        n, layout = weight_layout(p, x.shape[1])
        arr[i] = Projection(x.data_ptr(), p.data_ptr(), s.data_ptr(), y.data_ptr(),
                            n, x.shape[1], layout, 0,
                            b.data_ptr() if b is not None else 0,
                            r.data_ptr() if r is not None else 0)
    return arr


def forward_grouped_workspace_bytes(m: int, shapes: Sequence[tuple]) -> int:
    arr = (Projection * len(shapes))()
    for i, (n, k) in enumerate(shapes):
        arr[i] = Projection(0, 0, 0, 0, n, k)
    return int(_lib.bitlinear_forward_grouped_workspace_bytes(len(shapes), arr, m))


def forward_grouped_launches(m: int, shapes: Sequence[tuple]) -> int:
    """Kernels a grouped forward over projections of these (N, K) enqueues."""
    arr = (Projection * len(shapes))()
    for i, (n, k) in enumerate(shapes):
        arr[i] = Projection(0, 0, 0, 0, n, k)
    return int(_lib.bitlinear_forward_grouped_launches(len(shapes), arr, m))


class GroupedCall:
    """A prepared grouped forward: descriptors and workspace built once, so
    repeated calls only enqueue the kernels.  Optional per projection: a
    bf16 bias [N] and a bf16 residual [M, N] (may be that projection's
    output, for an in-place add)."""

    def __init__(self, xs, packeds, w_scales, outs=None, workspace=None, biases=None,
                 residuals=None):
        if not (len(xs) == len(packeds) == len(w_scales)) or not xs:
            raise ValueError("xs, packeds and w_scales must be non-empty lists of one length")
        m = xs[0].shape[0]
        dev = xs[0].device
        for x, p, s in zip(xs, packeds, w_scales):
            _require(x, torch.bfloat16, 2, "x", device=dev)
            _require(p, torch.uint8, 2, "packed", device=dev)
            _require_scale(s, dev)
            if x.shape[0] != m:
                raise ValueError("inconsistent token counts in grouped call")
            weight_layout(p, x.shape[1])
        if outs is None:
            outs = [torch.empty((m, weight_layout(p, x.shape[1])[0]), dtype=torch.bfloat16,
                                device=x.device) for x, p in zip(xs, packeds)]
        if len(outs) != len(xs):
            raise ValueError("one output per projection")
        for x, p, y in zip(xs, packeds, outs):
            _require(y, torch.bfloat16, 2, "out", shape=(m, weight_layout(p, x.shape[1])[0]),
                     device=dev)
        for lst, what in ((biases, "biases"), (residuals, "residuals")):
            if lst is not None and len(lst) != len(xs):
                raise ValueError(f"{what}: one entry (or None) per projection")
        for i, (x, p) in enumerate(zip(xs, packeds)):
            n = weight_layout(p, x.shape[1])[0]
            if biases is not None and biases[i] is not None:
                _require(biases[i], torch.bfloat16, 1, "bias", shape=(n,), device=dev)
            if residuals is not None and residuals[i] is not None:
                _require(residuals[i], torch.bfloat16, 2, "residual", shape=(m, n), device=dev)
        self.m = m
        self.outs = outs
        self._keep = (list(xs), list(packeds), list(w_scales), outs, biases, residuals)
        self._arr = _projections(xs, packeds, w_scales, outs, biases, residuals)
        need = int(_lib.bitlinear_forward_grouped_workspace_bytes(len(xs), self._arr, m))
        self.workspace = _workspace(need, xs[0].device, workspace)
        self._dev = xs[0]

    def __call__(self, stream=None):
        _launch(_lib.bitlinear_forward_grouped,
                (len(self._arr), self._arr, self.m, _ptr(self.workspace), _nbytes(self.workspace)),
                self._dev.device, stream)
        return self.outs


def forward_grouped(xs, packeds, w_scales, outs=None, workspace=None):
    """Independent BitLinear forwards with one token count, one pass."""
    return GroupedCall(xs, packeds, w_scales, outs, workspace)()


def forward_grouped_inspect(xs, packeds, w_scales, wait_polls: int = 0):
    """bitlinear_forward_grouped_inspect: the grouped forward, plus what its
    kernels computed on the way.  Returns (ys, inspections, status) where
    inspections[i] is a dict of the int8 codes [M, K], fp32 scales [M], int32
    code sums [M] and int32 accumulators [M, N] of projection i, and status
    is the device int32 status word (1: a decode wait gave up)."""
    call = GroupedCall(xs, packeds, w_scales)
    m, dev = call.m, call._dev.device
    ins = (Inspect * len(xs))()
    keep = []
    for i, (x, y) in enumerate(zip(xs, call.outs)):
        d = {"q": torch.empty((m, x.shape[1]), dtype=torch.int8, device=dev),
             "x_scale": torch.empty(max(m, 4), dtype=torch.float32, device=dev)[:m],
             "qsum": torch.empty(max(m, 4), dtype=torch.int32, device=dev)[:m],
             "acc": torch.empty((m, y.shape[1]), dtype=torch.int32, device=dev)}
        ins[i] = Inspect(d["q"].data_ptr(), d["x_scale"].data_ptr(), d["qsum"].data_ptr(),
                         d["acc"].data_ptr())
        keep.append(d)
    status = torch.zeros(4, dtype=torch.int32, device=dev)
    _launch(_lib.bitlinear_forward_grouped_inspect,
            (len(xs), call._arr, m, ins, _ptr(status), int(wait_polls), _ptr(call.workspace),
             _nbytes(call.workspace)), dev)
    return call.outs, keep, status[:1]


def forward_acc(q: torch.Tensor, packed: torch.Tensor, out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None):
    """Exact int32 accumulators q . u^T for caller-supplied int8 codes;
    `packed` in either layout."""
    _require(q, torch.int8, 2, "q")
    _require(packed, torch.uint8, 2, "packed", device=q.device)
    m, k = q.shape
    n, layout = weight_layout(packed, k)
    if out is None:
        out = torch.empty((m, n), dtype=torch.int32, device=q.device)
    _require(out, torch.int32, 2, "out", shape=(m, n), device=q.device)
    ws = _workspace(forward_workspace_bytes(m, n, k), q.device, workspace)
    fn = _lib.bitlinear_forward_acc_tiled if layout == LAYOUT_TILED else _lib.bitlinear_forward_acc
    _launch(fn, (m, n, k, _ptr(q), _ptr(packed), _ptr(out), _ptr(ws), _nbytes(ws)), q.device)
    return out


class BitLinear:
    """Inference-time BitLinear layer: packs fp32 latent weights once, then
    runs the forward pass on bf16 activations, adding the bf16 bias if one is
    given (as nn.Linear's).  The weights are kept in the tiled layout when the
    shape allows it (N % 16 == 0, K % 256 == 0) unless tiled=False; `packed`
    holds them in that layout."""

    def __init__(self, weight: torch.Tensor, bias: torch.Tensor | None = None,
                 tiled: bool = True):
        self.out_features, self.in_features = weight.shape
        self.packed, self.w_scale = pack_weights(weight.contiguous())
        if tiled and self.out_features % 16 == 0 and self.in_features % 256 == 0:
            self.packed = tile_weights(self.packed)
        self.bias = None if bias is None else bias.to(torch.bfloat16).contiguous()

    def __call__(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> torch.Tensor:
        """y = BitLinear(x) (+ bias); with `residual` (same shape as y), y +
        residual, added in the same pass."""
        lead = x.shape[:-1]
        res = None if residual is None else residual.reshape(-1, self.out_features).contiguous()
        y = forward(x.reshape(-1, self.in_features).contiguous(), self.packed, self.w_scale,
                    bias=self.bias, residual=res)
        return y.reshape(*lead, self.out_features)


# --------------------------------------------------------------------------
# Operators around the product (include/bitlinear_layer.h)

WEIGHT_NONE, WEIGHT_BF16, WEIGHT_F32 = 0, 1, 2  # BL_WEIGHT_*


def _need(t, dtype, name, shape, device):
    """_require of a tensor of a known shape and device, quickly when it fits."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and
            t.device == device and t.is_contiguous()):
        _require(t, dtype, len(shape), name, shape, device)


def _norm_weight(weight, k, device):
    """BL_WEIGHT_* of a norm's weight (bf16 or fp32 [K], or None)."""
    if weight is None:
        return WEIGHT_NONE
    if not isinstance(weight, torch.Tensor) or weight.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("weight must be a bfloat16 or float32 tensor, or None")
    _require(weight, weight.dtype, 1, "weight", shape=(k,), device=device)
    return WEIGHT_BF16 if weight.dtype == torch.bfloat16 else WEIGHT_F32


def _opt(t: torch.Tensor | None):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _rows_f32(m: int, device) -> torch.Tensor:
    return torch.empty(max(m, 4), dtype=torch.float32, device=device)[:m]


class Normed(NamedTuple):
    """What a NormQuantCall writes: int8 codes [M, K] and scales [M] of the
    norm's output, the residual stream h [M, K] (x itself without a residual),
    1 / rms per row [M], and the norm's bf16 output n [M, K] (None unless
    asked for)."""
    q: torch.Tensor
    x_scale: torch.Tensor
    h: torch.Tensor
    rstd: torch.Tensor
    n: torch.Tensor | None


class NormQuantCall:
    """A prepared bitlinear_rms_norm_quant: h = bf16(x + residual), RMSNorm of
    h with an optional bf16 or fp32 weight [K], and the int8 codes and scales
    of its output.  Outputs are allocated once (or given as `out`, a Normed;
    its h may be x or the residual, for an update in place); each call only
    enqueues the kernel."""

    def __init__(self, x, weight=None, residual=None, eps: float = 1e-6, want_norm: bool = False,
                 out: Normed | None = None):
        _require(x, torch.bfloat16, 2, "x")
        (m, k), dev = x.shape, x.device
        wtype = _norm_weight(weight, k, dev)
        if residual is not None:
            _require(residual, torch.bfloat16, 2, "residual", shape=(m, k), device=dev)
        if out is None:
            out = Normed(torch.empty((m, k), dtype=torch.int8, device=dev), _rows_f32(m, dev),
                         x if residual is None else torch.empty_like(x), _rows_f32(m, dev),
                         torch.empty_like(x) if want_norm else None)
        _require(out.q, torch.int8, 2, "out.q", shape=(m, k), device=dev)
        _require(out.x_scale, torch.float32, 1, "out.x_scale", shape=(m,), device=dev)
        _require(out.h, torch.bfloat16, 2, "out.h", shape=(m, k), device=dev)
        _require(out.rstd, torch.float32, 1, "out.rstd", shape=(m,), device=dev)
        if out.n is not None:
            _require(out.n, torch.bfloat16, 2, "out.n", shape=(m, k), device=dev)
        self.out = out
        self._dev, self._keep = dev, (x, weight, residual)
        # without a residual h is x: nothing to write unless it goes elsewhere
        h = None if residual is None and out.h.data_ptr() == x.data_ptr() else out.h
        self._args = (m, k, _ptr(x), _opt(residual), _opt(weight), wtype, float(eps), _opt(h),
                      _ptr(out.rstd), _opt(out.n), _ptr(out.q), _ptr(out.x_scale))

    def __call__(self, stream=None) -> Normed:
        _launch(_lib.bitlinear_rms_norm_quant, self._args, self._dev, stream)
        return self.out


def rms_norm_quant(x, weight=None, residual=None, eps: float = 1e-6, want_norm: bool = False) -> Normed:
    """Residual add, RMSNorm and int8 codes of its output, one kernel (see
    NormQuantCall)."""
    return NormQuantCall(x, weight, residual, eps, want_norm)()


class NormQuantBackwardCall:
    """A prepared gradient of rms_norm_quant.  dn: bf16 gradient [M, K] of the
    norm's output (the codes pass it straight through); h, rstd: what the
    forward wrote; dh: bf16 gradient of h, or None.  A call returns (dx,
    dweight): dx bf16 [M, K] is the gradient of x and of the residual, dweight
    fp32 [K] that of the weight (None without a weight, and with want_dweight
    False, for a frozen one); with accumulate it is added to the given
    `dweight`."""

    def __init__(self, dn, h, rstd, weight=None, dh=None, dx=None, dweight=None,
                 accumulate: bool = False, workspace=None, want_dweight: bool = True):
        _require(dn, torch.bfloat16, 2, "dn")
        (m, k), dev = dn.shape, dn.device
        _require(h, torch.bfloat16, 2, "h", shape=(m, k), device=dev)
        _require(rstd, torch.float32, 1, "rstd", shape=(m,), device=dev)
        wtype = _norm_weight(weight, k, dev)
        if dh is not None:
            _require(dh, torch.bfloat16, 2, "dh", shape=(m, k), device=dev)
        if accumulate and dweight is None:
            raise ValueError("accumulate needs the dweight to add to")
        if dweight is not None and not want_dweight:
            raise ValueError("a dweight is given and want_dweight is False")
        if dx is None:
            dx = torch.empty_like(dn)
        _require(dx, torch.bfloat16, 2, "dx", shape=(m, k), device=dev)
        if dweight is None and weight is not None and want_dweight:
            dweight = torch.empty(k, dtype=torch.float32, device=dev)
        if dweight is not None:
            _require(dweight, torch.float32, 1, "dweight", shape=(k,), device=dev)
        need = int(_lib.bitlinear_rms_norm_quant_backward_workspace_bytes(m, k, dweight is not None))
        self.workspace = _workspace(need, dev, workspace)
        self.dx, self.dweight = dx, dweight
        self._dev, self._keep = dev, (dn, h, rstd, weight, dh)
        self._args = (m, k, _ptr(dn), _ptr(h), _ptr(rstd), _opt(weight), wtype, _opt(dh), _ptr(dx),
                      _opt(dweight), int(accumulate), _ptr(self.workspace), _nbytes(self.workspace))

    def __call__(self, stream=None):
        _launch(_lib.bitlinear_rms_norm_quant_backward, self._args, self._dev, stream)
        return self.dx, self.dweight


def rms_norm_quant_backward(dn, h, rstd, weight=None, dh=None, want_dweight: bool = True):
    """(dx, dweight) of rms_norm_quant (see NormQuantBackwardCall)."""
    return NormQuantBackwardCall(dn, h, rstd, weight, dh, want_dweight=want_dweight)()


def restore_activations(q: torch.Tensor, x_scale: torch.Tensor,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """The activations that int8 codes [M, K] and scales [M] stand for:
    bf16(q / x_scale)."""
    _require(q, torch.int8, 2, "q")
    shape, dev = q.shape, q.device
    _need(x_scale, torch.float32, "x_scale", shape[:1], dev)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    else:
        _need(out, torch.bfloat16, "out", shape, dev)
    _launch(_lib.bitlinear_restore_activations,
            (*shape, q.data_ptr(), x_scale.data_ptr(), out.data_ptr()), dev)
    return out


class GroupedQuantizedCall:
    """A prepared grouped forward on int8 activations: per projection the codes
    [M, K] and scales [M] (of rms_norm_quant or act_quant; projections may share
    them), the packed weights in either layout and their scale, and optionally a
    bf16 bias [N] and residual [M, N] (may be the output).  Results are those of
    GroupedCall on the bf16 activations behind the codes (which is the faster
    one at up to 4 tokens, where it quantizes inside its one kernel)."""

    def __init__(self, qs, x_scales, packeds, w_scales, outs=None, workspace=None, biases=None,
                 residuals=None):
        count = len(qs)
        if not (count == len(x_scales) == len(packeds) == len(w_scales)) or not count:
            raise ValueError("qs, x_scales, packeds and w_scales must be non-empty lists of one length")
        for lst, what in ((outs, "outs"), (biases, "biases"), (residuals, "residuals")):
            if lst is not None and len(lst) != count:
                raise ValueError(f"{what}: one entry per projection")
        _require(qs[0], torch.int8, 2, "q")
        m, dev = qs[0].shape[0], qs[0].device
        self._arr, self._codes = (Projection * count)(), (Codes * count)()
        self.outs = []
        for i, (q, xs, p, s) in enumerate(zip(qs, x_scales, packeds, w_scales)):
            _require(q, torch.int8, 2, "q", device=dev)
            k = q.shape[1]
            _need(q, torch.int8, "q", (m, k), dev)
            _need(xs, torch.float32, "x_scale", (m,), dev)
            _require(p, torch.uint8, 2, "packed", device=dev)
            _require_scale(s, dev)
            n, layout = weight_layout(p, k)
            y = outs[i] if outs is not None else torch.empty((m, n), dtype=torch.bfloat16, device=dev)
            _need(y, torch.bfloat16, "out", (m, n), dev)
            b = biases[i] if biases is not None else None
            r = residuals[i] if residuals is not None else None
            if b is not None:
                _need(b, torch.bfloat16, "bias", (n,), dev)
            if r is not None:
                _need(r, torch.bfloat16, "residual", (m, n), dev)
            self.outs.append(y)
            self._codes[i] = Codes(q.data_ptr(), xs.data_ptr())
            self._arr[i] = Projection(0, p.data_ptr(), s.data_ptr(), y.data_ptr(), n, k, layout, 0,
                                      0 if b is None else b.data_ptr(), 0 if r is None else r.data_ptr())
        need = int(_lib.bitlinear_forward_grouped_workspace_bytes(count, self._arr, m))
        self.workspace = _workspace(need, dev, workspace)
        self._dev = dev
        self._keep = (list(qs), list(x_scales), list(packeds), list(w_scales), biases, residuals)
        self._args = (count, self._arr, self._codes, m, _ptr(self.workspace), _nbytes(self.workspace))

    def __call__(self, stream=None):
        _launch(_lib.bitlinear_forward_grouped_quantized, self._args, self._dev, stream)
        return self.outs


def forward_quantized(q, x_scale, packed, w_scale, out=None, workspace=None, bias=None,
                      residual=None) -> torch.Tensor:
    """forward() on int8 activations: codes [M, K] and scales [M] (see
    GroupedQuantizedCall)."""
    return GroupedQuantizedCall([q], [x_scale], [packed], [w_scale], None if out is None else [out],
                                workspace, [bias], [residual])()[0]


class BackwardCall:
    """Prepared gradients of one BitLinear, from dy bf16 [M, N]: of its input
    (packed weights in either layout and their scale), dx bf16 [M, K], and of
    its latent weights (the input's int8 codes [M, K] and scales [M]: its 8-bit
    checkpoint), dw fp32 [N, K] and with `bias` dbias fp32 [N].  Leave `packed`
    out for no dx, or `q` for no dw.  `residual` (bf16 [M, K], may be dx) is
    added to dx, so that layers that share an input add their gradients up;
    with accumulate, dw and dbias are added to the given tensors.  Outputs and
    workspace are allocated once unless given; a call returns (dx, dw, dbias),
    None for what is left out."""

    def __init__(self, dy, q=None, x_scale=None, packed=None, w_scale=None, bias: bool = False,
                 k: int | None = None, residual=None, dx=None, dw=None, dbias=None,
                 accumulate: bool = False, workspace=None):
        _require(dy, torch.bfloat16, 2, "dy")
        (m, n), dev = dy.shape, dy.device
        if q is None and packed is None:
            raise ValueError("nothing to do: give packed (for dx) or q (for dw)")
        if q is not None:
            _require(q, torch.int8, 2, "q", device=dev)
            if k is not None and k != q.shape[1]:
                raise ValueError(f"q has {q.shape[1]} columns, k is {k}")
            k = q.shape[1]
            _require(q, torch.int8, 2, "q", shape=(m, k))
            _require(x_scale, torch.float32, 1, "x_scale", shape=(m,), device=dev)
            bias = bias or dbias is not None
            if accumulate and (dw is None or (bias and dbias is None)):
                raise ValueError("accumulate needs the tensors to add to")
            if dw is None:
                dw = torch.empty((n, k), dtype=torch.float32, device=dev)
            _require(dw, torch.float32, 2, "dw", shape=(n, k), device=dev)
            if bias and dbias is None:
                dbias = _rows_f32(n, dev)
            if dbias is not None:
                _require(dbias, torch.float32, 1, "dbias", shape=(n,), device=dev)
        elif dw is not None or dbias is not None or bias:
            raise ValueError("dw and dbias need q and x_scale")
        layout = LAYOUT_ROWS
        if packed is not None:
            _require(packed, torch.uint8, 2, "packed", device=dev)
            _require_scale(w_scale, dev)
            if k is None:
                k = 4 * packed.shape[1]
            rows, layout = weight_layout(packed, k)
            if rows != n:
                raise ValueError(f"packed weights have {rows} rows, dy {n} columns")
            if residual is not None:
                _require(residual, torch.bfloat16, 2, "residual", shape=(m, k), device=dev)
            if dx is None:
                dx = torch.empty((m, k), dtype=torch.bfloat16, device=dev)
            _require(dx, torch.bfloat16, 2, "dx", shape=(m, k), device=dev)
        elif dx is not None or residual is not None:
            raise ValueError("dx needs packed and w_scale")
        need = int(_lib.bitlinear_backward_workspace_bytes(m, n, k, dx is not None, dw is not None))
        self.workspace = _workspace(need, dev, workspace)
        self._out = (dx, dw, dbias)
        self._dev, self._keep = dev, (dy, q, x_scale, packed, w_scale, residual)
        self._args = (m, n, k, _ptr(dy), _opt(packed), layout, _opt(w_scale), _opt(residual),
                      _opt(dx), _opt(q), _opt(x_scale), _opt(dw), _opt(dbias), int(accumulate),
                      _ptr(self.workspace), _nbytes(self.workspace))

    def __call__(self, stream=None):
        _launch(_lib.bitlinear_backward, self._args, self._dev, stream)
        return self._out


def backward_input(dy, packed, w_scale, k: int | None = None, residual=None, out=None,
                   workspace=None) -> torch.Tensor:
    """Gradient of BitLinear's input, bf16 [M, K] (see BackwardCall; give K for
    tiled weights)."""
    return BackwardCall(dy, None, None, packed, w_scale, k=k, residual=residual, dx=out,
                        workspace=workspace)()[0]


def backward_weight(dy, q, x_scale, bias: bool = False, out=None, dbias=None,
                    accumulate: bool = False, workspace=None):
    """Gradients of BitLinear's latent weights, fp32 [N, K], and of its bias,
    fp32 [N] (None unless `bias`; see BackwardCall)."""
    return BackwardCall(dy, q, x_scale, bias=bias, dw=out, dbias=dbias, accumulate=accumulate,
                        workspace=workspace)()[1:]


class W4Weights(NamedTuple):
    """4-bit weights of an [N, K] matrix with a bf16 scale per row and group of
    `group` consecutive K (the storage of bitlinear_layer.h): codes uint8
    [N/16, K/128, 4, 16, 16], scales bf16 [N/16, K/group, 16], both with N and
    K rounded up to whole blocks."""
    codes: torch.Tensor
    scales: torch.Tensor
    n: int
    k: int
    group: int


def _require_w4(w: W4Weights, device=None):
    if w.n < 1 or w.k < 1 or w.group < 1 or w.k % w.group:
        raise ValueError("W4Weights: n, k and group must be positive and group divide k")
    nb, kt = (w.n + 15) // 16, (w.k + 127) // 128
    _require(w.codes, torch.uint8, 5, "codes", shape=(nb, kt, 4, 16, 16), device=device)
    _require(w.scales, torch.bfloat16, 3, "scales", shape=(nb, w.k // w.group, 16),
             device=w.codes.device)


def pack_weights_w4(w: torch.Tensor, group: int = 128) -> W4Weights:
    """Latent fp32 weights [N, K] -> 4-bit codes and group scales.  group: a
    power of two from 32 to 1024 that divides K."""
    _require(w, torch.float32, 2, "w")
    n, k = w.shape
    if group < 32 or group > 1024 or group & (group - 1) or k % group:
        raise ValueError("group must be a power of two from 32 to 1024 that divides K")
    out = W4Weights(torch.empty(((n + 15) // 16, (k + 127) // 128, 4, 16, 16), dtype=torch.uint8,
                                device=w.device),
                    torch.empty(((n + 15) // 16, k // group, 16), dtype=torch.bfloat16,
                                device=w.device), n, k, group)
    _launch(_lib.bitlinear_w4_pack, (_ptr(w), n, k, group, _ptr(out.codes), _ptr(out.scales)),
            w.device)
    return out


def unpack_weights_w4(w: W4Weights) -> torch.Tensor:
    """The fp32 weights [N, K] that 4-bit codes and scales stand for."""
    _require_w4(w)
    out = torch.empty((w.n, w.k), dtype=torch.float32, device=w.codes.device)
    _launch(_lib.bitlinear_w4_unpack,
            (_ptr(w.codes), _ptr(w.scales), w.n, w.k, w.group, _ptr(out)), w.codes.device)
    return out


class W4Call:
    """A prepared product of int8 activations (codes [M, K], scales [M]) with
    4-bit weights: y bf16 [M, N], with an optional bf16 bias [N].  Made for up to
    16 tokens: every 16 read the weights again."""

    def __init__(self, q, x_scale, w: W4Weights, out=None, bias=None):
        _require(q, torch.int8, 2, "q")
        (m, k), dev = q.shape, q.device
        _require(x_scale, torch.float32, 1, "x_scale", shape=(m,), device=dev)
        _require_w4(w, dev)
        if k != w.k:
            raise ValueError(f"q has {k} columns, the weights {w.k}")
        if bias is not None:
            _require(bias, torch.bfloat16, 1, "bias", shape=(w.n,), device=dev)
        if out is None:
            out = torch.empty((m, w.n), dtype=torch.bfloat16, device=dev)
        _require(out, torch.bfloat16, 2, "out", shape=(m, w.n), device=dev)
        self.out = out
        self._dev, self._keep = dev, (q, x_scale, w, bias)
        self._args = (m, w.n, k, w.group, _ptr(q), _ptr(x_scale), _ptr(w.codes), _ptr(w.scales),
                      _opt(bias), _ptr(out))

    def __call__(self, stream=None) -> torch.Tensor:
        _launch(_lib.bitlinear_w4_forward, self._args, self._dev, stream)
        return self.out


def forward_w4(q, x_scale, w: W4Weights, out=None, bias=None) -> torch.Tensor:
    """y = (codes / x_scale) . weights^T as bf16 [M, N] (see W4Call)."""
    return W4Call(q, x_scale, w, out, bias)()


# --------------------------------------------------------------------------
# Operators of a feed-forward block and of a training step (include/bitlinear_ffn.h)

class W8Weights(NamedTuple):
    """8-bit weights of an [N, K] matrix with an fp32 scale per row (the storage
    of bitlinear_ffn.h): codes int8 [N/16, K/64, 4, 16, 16], N and K rounded up
    to whole blocks; scale fp32 [N]."""
    codes: torch.Tensor
    scale: torch.Tensor
    n: int
    k: int


def _require_w8(w: W8Weights, device=None):
    if w.n < 1 or w.k < 1:
        raise ValueError("W8Weights: n and k must be positive")
    _require(w.codes, torch.int8, 5, "codes", shape=((w.n + 15) // 16, (w.k + 63) // 64, 4, 16, 16), device=device)
    _require(w.scale, torch.float32, 1, "scale", shape=(w.n,), device=w.codes.device)


def pack_weights_w8(w: torch.Tensor) -> W8Weights:
    """Latent fp32 weights [N, K] -> 8-bit codes and a scale per row."""
    _require(w, torch.float32, 2, "w")
    n, k = w.shape
    out = W8Weights(torch.empty(((n + 15) // 16, (k + 63) // 64, 4, 16, 16), dtype=torch.int8, device=w.device),
                    _rows_f32(n, w.device), n, k)
    _launch(_lib.bitlinear_w8_pack, (_ptr(w), n, k, _ptr(out.codes), _ptr(out.scale)), w.device)
    return out


def unpack_weights_w8(w: W8Weights) -> torch.Tensor:
    """The fp32 weights [N, K] that 8-bit codes and scales stand for."""
    _require_w8(w)
    out = torch.empty((w.n, w.k), dtype=torch.float32, device=w.codes.device)
    _launch(_lib.bitlinear_w8_unpack, (_ptr(w.codes), _ptr(w.scale), w.n, w.k, _ptr(out)), w.codes.device)
    return out


class W8Call:
    """A prepared product of int8 activations (codes [M, K], scales [M]) with
    8-bit weights: y bf16 [M, N], with an optional bf16 bias [N].  For any number
    of tokens."""

    def __init__(self, q, x_scale, w: W8Weights, out=None, bias=None, workspace=None):
        _require(q, torch.int8, 2, "q")
        (m, k), dev = q.shape, q.device
        _require(x_scale, torch.float32, 1, "x_scale", shape=(m,), device=dev)
        _require_w8(w, dev)
        if k != w.k:
            raise ValueError(f"q has {k} columns, the weights {w.k}")
        if bias is not None:
            _require(bias, torch.bfloat16, 1, "bias", shape=(w.n,), device=dev)
        if out is None:
            out = torch.empty((m, w.n), dtype=torch.bfloat16, device=dev)
        _require(out, torch.bfloat16, 2, "out", shape=(m, w.n), device=dev)
        self.workspace = _workspace(int(_lib.bitlinear_w8_forward_workspace_bytes(m, w.n, k)), dev, workspace)
        self.out = out
        self._dev, self._keep = dev, (q, x_scale, w, bias)
        self._args = (m, w.n, k, _ptr(q), _ptr(x_scale), _ptr(w.codes), _ptr(w.scale), _opt(bias), _ptr(out),
                      _ptr(self.workspace), _nbytes(self.workspace))

    def __call__(self, stream=None) -> torch.Tensor:
        _launch(_lib.bitlinear_w8_forward, self._args, self._dev, stream)
        return self.out


def forward_w8(q, x_scale, w: W8Weights, out=None, bias=None, workspace=None) -> torch.Tensor:
    """y = (codes / x_scale) . weights^T as bf16 [M, N] (see W8Call)."""
    return W8Call(q, x_scale, w, out, bias, workspace)()


# --------------------------------------------------------------------------
# Gated feed-forward block

ACTIVATIONS = {"relu2": 1, "silu": 2}  # BL_ACT_*: max(g, 0)^2, g / (1 + exp(-g))


def _activation(name) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {name!r}")
    return ACTIVATIONS[name]


class GatedWeights(NamedTuple):
    """Ternary weights of a feed-forward block's gate and up projections, [N, K]
    each, laid out for GatedCall (the storage of bitlinear_ffn.h): codes uint8
    [N/16, K/256, 2, 4, 16, 16], N and K rounded up to whole blocks; the two
    weight scales fp32 [1]."""
    codes: torch.Tensor
    gate_scale: torch.Tensor
    up_scale: torch.Tensor
    n: int
    k: int


def gated_weights(gate, gate_scale, up, up_scale, k: int | None = None) -> GatedWeights:
    """Packed ternary weights of the gate and up projections, each in either
    layout (give K for tiled ones), laid out for GatedCall."""
    _require(gate, torch.uint8, 2, "gate")
    dev = gate.device
    _require(up, torch.uint8, 2, "up", device=dev)
    _require_scale(gate_scale, dev, "gate_scale")
    _require_scale(up_scale, dev, "up_scale")
    if k is None:
        k = 4 * gate.shape[1]
    (n, lg), (nu, lu) = weight_layout(gate, k), weight_layout(up, k)
    if n != nu:
        raise ValueError(f"the gate has {n} outputs, the up projection {nu}")
    codes = torch.empty(((n + 15) // 16, (k + 255) // 256, 2, 4, 16, 16), dtype=torch.uint8, device=dev)
    _launch(_lib.bitlinear_gated_weights, (n, k, _ptr(gate), lg, _ptr(up), lu, _ptr(codes)), dev)
    return GatedWeights(codes, gate_scale, up_scale, n, k)


class Gated(NamedTuple):
    """What a GatedCall writes: a = act(g) * u, and where they are kept g and u
    themselves, bf16 [M, N] each."""
    a: torch.Tensor
    g: torch.Tensor | None
    u: torch.Tensor | None


class GatedCall:
    """A prepared gated feed-forward entry: both projections of int8 activations
    (codes [M, K], scales [M]), the activation function ("relu2" or "silu") and
    the product, in one kernel.  `keep` also writes g and u, which the gradients
    read.  Outputs (or `out`, a Gated) and workspace are allocated once."""

    def __init__(self, q, x_scale, w: GatedWeights, activation: str, keep: bool = False, out: Gated | None = None,
                 workspace=None):
        _require(q, torch.int8, 2, "q")
        (m, k), dev, act = q.shape, q.device, _activation(activation)
        _require(x_scale, torch.float32, 1, "x_scale", shape=(m,), device=dev)
        if w.n < 1 or w.k < 1:
            raise ValueError("GatedWeights: n and k must be positive")
        _require(w.codes, torch.uint8, 6, "codes", shape=((w.n + 15) // 16, (w.k + 255) // 256, 2, 4, 16, 16),
                 device=dev)
        _require_scale(w.gate_scale, dev, "gate_scale")
        _require_scale(w.up_scale, dev, "up_scale")
        if k != w.k:
            raise ValueError(f"q has {k} columns, the weights {w.k}")
        if out is None:
            out = Gated(*(torch.empty((m, w.n), dtype=torch.bfloat16, device=dev) if i == 0 or keep else None
                          for i in range(3)))
        _require(out.a, torch.bfloat16, 2, "out.a", shape=(m, w.n), device=dev)
        if (out.g is None) != (out.u is None) or (keep and out.g is None):
            raise ValueError("out.g and out.u are kept together (and needed with keep)")
        for t, name in ((out.g, "out.g"), (out.u, "out.u")):
            if t is not None:
                _require(t, torch.bfloat16, 2, name, shape=(m, w.n), device=dev)
        self.workspace = _workspace(int(_lib.bitlinear_gated_forward_workspace_bytes(m, w.n, k)), dev, workspace)
        self.out = out
        self._dev, self._keep = dev, (q, x_scale, w)
        self._args = (m, w.n, k, _ptr(q), _ptr(x_scale), _ptr(w.codes), _ptr(w.gate_scale), _ptr(w.up_scale), act,
                      _ptr(out.a), _opt(out.g), _opt(out.u), _ptr(self.workspace), _nbytes(self.workspace))

    def __call__(self, stream=None) -> Gated:
        _launch(_lib.bitlinear_gated_forward, self._args, self._dev, stream)
        return self.out


def forward_gated(q, x_scale, w: GatedWeights, activation: str, keep: bool = False) -> Gated:
    """The gate and up projections, the activation function and the product (see
    GatedCall)."""
    return GatedCall(q, x_scale, w, activation, keep)()


class GatedBackwardCall:
    """Prepared gradients of a gated feed-forward entry, from da bf16 [M, N] and
    the g and u that the forward kept: of the input (packed weights of both
    projections, each in either layout, and their scales), dx bf16 [M, K], and of
    both latent weights (the input's int8 codes and scales), dw_gate and dw_up
    fp32 [N, K].  Leave `gate` and `up` out for no dx, or `q` for no weights'
    gradients.  `residual` (bf16 [M, K], may be dx) is added to dx; with
    accumulate the weights' gradients are added to the given tensors.  A call
    returns (dx, dw_gate, dw_up), None for what is left out."""

    def __init__(self, da, g, u, activation: str, q=None, x_scale=None, gate=None, gate_scale=None, up=None,
                 up_scale=None, k: int | None = None, residual=None, dx=None, dw_gate=None, dw_up=None,
                 accumulate: bool = False, workspace=None):
        _require(da, torch.bfloat16, 2, "da")
        (m, n), dev, act = da.shape, da.device, _activation(activation)
        _require(g, torch.bfloat16, 2, "g", shape=(m, n), device=dev)
        _require(u, torch.bfloat16, 2, "u", shape=(m, n), device=dev)
        if (gate is None) != (up is None):
            raise ValueError("gate and up are given together")
        if q is None and gate is None:
            raise ValueError("nothing to do: give gate and up (for dx) or q (for the weights' gradients)")
        if q is not None:
            _require(q, torch.int8, 2, "q", device=dev)
            if k is not None and k != q.shape[1]:
                raise ValueError(f"q has {q.shape[1]} columns, k is {k}")
            k = q.shape[1]
            _require(q, torch.int8, 2, "q", shape=(m, k))
            _require(x_scale, torch.float32, 1, "x_scale", shape=(m,), device=dev)
            if (dw_gate is None) != (dw_up is None):
                raise ValueError("dw_gate and dw_up are given together")
            if accumulate and dw_gate is None:
                raise ValueError("accumulate needs the tensors to add to")
            if dw_gate is None:
                dw_gate, dw_up = (torch.empty((n, k), dtype=torch.float32, device=dev) for _ in range(2))
            _require(dw_gate, torch.float32, 2, "dw_gate", shape=(n, k), device=dev)
            _require(dw_up, torch.float32, 2, "dw_up", shape=(n, k), device=dev)
        elif dw_gate is not None or dw_up is not None:
            raise ValueError("dw_gate and dw_up need q and x_scale")
        lg = lu = LAYOUT_ROWS
        if gate is not None:
            _require(gate, torch.uint8, 2, "gate", device=dev)
            _require(up, torch.uint8, 2, "up", device=dev)
            _require_scale(gate_scale, dev, "gate_scale")
            _require_scale(up_scale, dev, "up_scale")
            if k is None:
                k = 4 * gate.shape[1]
            (ng, lg), (nu, lu) = weight_layout(gate, k), weight_layout(up, k)
            if ng != n or nu != n:
                raise ValueError(f"the packed weights have {ng} and {nu} rows, da {n} columns")
            if residual is not None:
                _require(residual, torch.bfloat16, 2, "residual", shape=(m, k), device=dev)
            if dx is None:
                dx = torch.empty((m, k), dtype=torch.bfloat16, device=dev)
            _require(dx, torch.bfloat16, 2, "dx", shape=(m, k), device=dev)
        elif dx is not None or residual is not None:
            raise ValueError("dx needs gate and up")
        need = int(_lib.bitlinear_gated_backward_workspace_bytes(m, n, k, dx is not None, dw_gate is not None))
        self.workspace = _workspace(need, dev, workspace)
        self._out = (dx, dw_gate, dw_up)
        self._dev, self._keep = dev, (da, g, u, q, x_scale, gate, gate_scale, up, up_scale, residual)
        self._args = (m, n, k, act, _ptr(da), _ptr(g), _ptr(u), _opt(gate), lg, _opt(up), lu, _opt(gate_scale),
                      _opt(up_scale), _opt(residual), _opt(dx), _opt(q), _opt(x_scale), _opt(dw_gate), _opt(dw_up),
                      int(accumulate), _ptr(self.workspace), _nbytes(self.workspace))

    def __call__(self, stream=None):
        _launch(_lib.bitlinear_gated_backward, self._args, self._dev, stream)
        return self._out


# --------------------------------------------------------------------------
# Gradient norm and clipping

GRAD_BF16, GRAD_F32 = 1, 2  # BL_GRAD_*


def _dense(t: torch.Tensor) -> bool:
    """Whether t's elements fill its piece of memory, in some order of its
    dimensions."""
    want = 1
    for stride, size in sorted((st, sz) for st, sz in zip(t.stride(), t.shape) if sz != 1):
        if stride != want and t.numel():
            return False
        want *= size
    return True


def _gradients(grads, outs):
    """Descriptors of the gradients, and their device."""
    if not grads:
        raise ValueError("at least one gradient")
    if outs is not None and len(outs) != len(grads):
        raise ValueError("outs: one tensor per gradient")
    arr = (Gradient * len(grads))()
    dev = grads[0].device if isinstance(grads[0], torch.Tensor) else None
    for i, g in enumerate(grads):
        o = g if outs is None else outs[i]
        for t, name in ((g, "a gradient"), (o, "an output")):
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise TypeError(f"{name} must be a CUDA (HIP) tensor")
            if t.dtype not in (torch.float32, torch.bfloat16):
                raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
            if t.device != dev:
                raise ValueError(f"{name} is on {t.device}, expected {dev}")
            if not _dense(t):
                raise ValueError(f"{name} must fill its memory (a slice of a larger tensor does not)")
        if o is not g and (o.shape != g.shape or o.dtype != g.dtype or (o.numel() > 1 and o.stride() != g.stride())):
            raise ValueError("an output must have its gradient's shape, type and strides")
        arr[i] = Gradient(g.data_ptr(), o.data_ptr(), g.numel(), GRAD_BF16 if g.dtype == torch.bfloat16 else GRAD_F32, 0)
    return arr, dev


class GradNormCall:
    """A prepared norm of many gradients together (fp32 or bf16 tensors of any
    shapes on one device): fp32 [1], on the device."""

    def __init__(self, grads, workspace=None):
        grads = list(grads)  # once: what a generator made is held by this list alone
        self._arr, self._dev = _gradients(grads, None)
        self.norm = _rows_f32(1, self._dev)
        need = int(_lib.bitlinear_grad_norm_workspace_bytes(len(self._arr), self._arr))
        self.workspace = _workspace(need, self._dev, workspace)
        self._keep = grads
        self._args = (len(self._arr), self._arr, _ptr(self.norm), _ptr(self.workspace), _nbytes(self.workspace))

    def __call__(self, stream=None) -> torch.Tensor:
        _launch(_lib.bitlinear_grad_norm, self._args, self._dev, stream)
        return self.norm


class ClipGradsCall:
    """Prepared clipping of many gradients to a norm of all of them together:
    each is multiplied by min(1, max_norm / (norm + 1e-6)), in place or into
    `outs`.  No gradient may be listed twice.  A call returns (norm, outs), norm
    fp32 [1] on the device: that before clipping.  Nothing waits for it: a norm
    that is not finite is the caller's to look at.  Autograd is told of the tensors
    that a call writes (not of a graph's replays), and so refuses to go back through
    a graph that has saved them."""

    def __init__(self, grads, max_norm: float, outs=None, workspace=None):
        grads = list(grads)
        max_norm = float(max_norm)
        if not max_norm >= 0:
            raise ValueError(f"max_norm must be 0 or more, got {max_norm}")
        self._arr, self._dev = _gradients(grads, outs)
        self.norm = _rows_f32(1, self._dev)
        need = int(_lib.bitlinear_grad_norm_workspace_bytes(len(self._arr), self._arr))
        self.workspace = _workspace(need, self._dev, workspace)
        self._keep = grads
        self.outs = grads if outs is None else list(outs)
        self._args = (len(self._arr), self._arr, max_norm, _ptr(self.norm), _ptr(self.workspace),
                      _nbytes(self.workspace))

    def __call__(self, stream=None):
        _launch(_lib.bitlinear_clip_gradients, self._args, self._dev, stream)
        torch.autograd.graph.increment_version(self.outs)
        return self.norm, self.outs


def grad_norm(grads) -> torch.Tensor:
    """The norm of all gradients together, fp32 [1] (see GradNormCall)."""
    return GradNormCall(grads)()


def clip_grads(grads, max_norm: float, outs=None):
    """(norm, clipped gradients), in place unless `outs` (see ClipGradsCall)."""
    return ClipGradsCall(grads, max_norm, outs)()
