"""Python binding of the fused normalization library (``libnormfuse.so``).

The functions here have the names of the C entry points declared in
``include/normfuse.h`` and only marshal arguments: torch tensors become
device pointers, the torch stream becomes a ``cudaStream_t``, and the return
status becomes an exception. The quantised calls that allocate their outputs
do so in C++ (``csrc/marshal.cc``) where that is built and the call is on the
current device and stream. Every step of the computation runs in the CUDA
kernels of the library; there is no fallback. If the library has not been
built, loading it raises.

PyTorch is used for device memory and streams only.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import importlib.machinery
import importlib.util
import os
import struct
import threading
from typing import NamedTuple

import torch

from .build import LIB_PATH, build as build_library, marshal_path

__all__ = [
    "LN_F32", "LN_BF16", "LN_F16", "LN_LAYERNORM", "LN_RMSNORM", "NormError",
    "LN_OK", "LN_ERR_NULL", "LN_ERR_ALIGN", "LN_ERR_SHAPE", "LN_ERR_UNSUPPORTED",
    "LN_ERR_CUDA", "LN_ERR_WORKSPACE", "LN_ERR_INVALID", "LN_ERR_SCRATCH_LIMIT",
    "LN_NOALLOC_SCRATCH_BYTES",
    "load_library", "build_library", "ln_fwd", "ln_fwd_ex", "ln_bwd", "ln_bwd_ex",
    "ln_bwd_workspace_bytes",
    "ln_status_string", "ln_last_cuda_error", "ln_device_error", "ln_bwd_noalloc",
    "ln_testing_select_kernels", "ln_testing_plan", "exported_symbols", "ln_fwd_from_partials",
    "LN_PARTIALS_SUM_SQ", "LN_PARTIALS_SUM_M2", "fused_norm_fwd_from_partials",
    "fused_norm_fwd", "fused_norm_bwd", "Workspace",
    "GN_ACT_NONE", "GN_ACT_SILU", "GN_ACT_GELU", "gn_fwd", "gn_bwd", "gn_workspace_bytes",
    "fused_group_norm_fwd", "fused_group_norm_bwd",
    "ROPE_HALF", "ROPE_INTERLEAVED", "rope_fwd", "rope_bwd", "rope_bwd_workspace_bytes",
    "rope_frequencies", "rope_axes", "fused_rope_fwd", "fused_rope_bwd",
    "MX_FP8_ROW", "MX_FP8_BLOCK", "MX_MXFP8", "MX_MXFP4", "MX_NVFP4", "Quantized",
    "quantized_empty", "mx_matrix_bytes", "mx_norm_fwd", "mx_quantize", "mx_dequantize",
    "mx_product", "fused_norm_quant_fwd", "quantize", "dequantize", "scaled_product",
]

# Mirrors of include/normfuse.h (a CPU test checks them against the header).
LN_F32, LN_BF16, LN_F16 = 0, 1, 2
LN_LAYERNORM, LN_RMSNORM = 0, 1
(LN_OK, LN_ERR_NULL, LN_ERR_ALIGN, LN_ERR_SHAPE, LN_ERR_UNSUPPORTED, LN_ERR_CUDA,
 LN_ERR_WORKSPACE, LN_ERR_INVALID, LN_ERR_SCRATCH_LIMIT) = range(9)
LN_NOALLOC_SCRATCH_BYTES = 16 << 20
LN_PARTIALS_SUM_SQ, LN_PARTIALS_SUM_M2 = 0, 1
_PARTIAL_CODES = {"sum_sq": LN_PARTIALS_SUM_SQ, "sum_m2": LN_PARTIALS_SUM_M2,
                  LN_PARTIALS_SUM_SQ: LN_PARTIALS_SUM_SQ, LN_PARTIALS_SUM_M2: LN_PARTIALS_SUM_M2}
_DTYPE_CODES = {torch.float32: LN_F32, torch.bfloat16: LN_BF16, torch.float16: LN_F16}
_MODE_CODES = {"layernorm": LN_LAYERNORM, "rmsnorm": LN_RMSNORM,
               LN_LAYERNORM: LN_LAYERNORM, LN_RMSNORM: LN_RMSNORM}

GN_ACT_NONE, GN_ACT_SILU, GN_ACT_GELU = 0, 1, 2
_ACT_CODES = {"none": GN_ACT_NONE, None: GN_ACT_NONE, "silu": GN_ACT_SILU, "gelu": GN_ACT_GELU,
              GN_ACT_NONE: GN_ACT_NONE, GN_ACT_SILU: GN_ACT_SILU, GN_ACT_GELU: GN_ACT_GELU}
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
_SCALING_CODES = {"none": 0, None: 0, "linear": 1, "ntk": 2, "yarn": 3}
# The C structs rope_heads, rope_heads_grad and rope_positions.
_ROPE_HEADS = struct.Struct("@PPPq3q3q")
_ROPE_HEADS_GRAD = struct.Struct("@PPPPPq3q3q3q")
_ROPE_POSITIONS = struct.Struct("@Piq3qPqif")
MX_FP8_ROW, MX_FP8_BLOCK, MX_MXFP8, MX_MXFP4, MX_NVFP4 = range(5)
_FORMAT_CODES = {"fp8_row": MX_FP8_ROW, "fp8_block": MX_FP8_BLOCK, "mxfp8": MX_MXFP8,
                 "mxfp4": MX_MXFP4, "nvfp4": MX_NVFP4}
# The C struct mx_matrix.
_MX_MATRIX = struct.Struct("@PPPiqq")

_lib = None
_marshal = None     # the binding's C++ part (csrc/marshal.cc), where it is built for this torch
_lock = threading.Lock()


class NormError(RuntimeError):
    """A non-zero ``ln_status`` returned by the library."""

    def __init__(self, status: int, where: str):
        self.status = status
        msg = ln_status_string(status)
        if status == 5:
            msg += f" (cudaError {ln_last_cuda_error()})"
        super().__init__(f"{where}: {msg}")


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load ``libnormfuse.so`` (built in-tree by ``build_library()``), or the one at
    ``path``. The binding's C++ part calls the same one; where it is not built for
    the torch that runs, its calls go through ctypes like all others."""
    global _lib, _marshal
    with _lock:
        if _lib is not None:
            return _lib
        path = path or LIB_PATH
        if not os.path.isfile(path):
            raise RuntimeError(
                f"CUDA library not built: {path} is missing. "
                "Run `python -m normalization_fwd_gb300.build` (needs nvcc).")
        lib = ctypes.CDLL(path)
        vp, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        ci = ctypes.c_int
        lib.ln_fwd.argtypes = [vp, vp, vp, vp, vp, f32, ci, ci, vp, vp, vp, vp, vp, vp,
                               i64, i64, ci]
        lib.ln_fwd.restype = ci
        lib.ln_fwd_ex.argtypes = [vp, vp, vp, vp, vp, f32, ci, ci, vp, vp, vp, vp, vp, vp, vp,
                                  vp, i64, i64, ci]
        lib.ln_fwd_ex.restype = ci
        lib.ln_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, ci, ci, ci,
                               vp, sz]
        lib.ln_bwd.restype = ci
        lib.ln_bwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, ci, ci, ci,
                                  vp, sz, ci]
        lib.ln_bwd_ex.restype = ci
        lib.ln_bwd_workspace_bytes.argtypes = [i64, i64, ci, ci, ctypes.POINTER(sz)]
        lib.ln_bwd_workspace_bytes.restype = ci
        lib.ln_status_string.argtypes = [ci]
        lib.ln_status_string.restype = ctypes.c_char_p
        lib.ln_last_cuda_error.argtypes = []
        lib.ln_last_cuda_error.restype = ci
        lib.ln_device_error.argtypes = [vp, ctypes.POINTER(ctypes.c_uint)]
        lib.ln_device_error.restype = ci
        lib.ln_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, ci, ci, ci]
        lib.ln_bwd_noalloc.restype = ci
        lib.ln_softmax_fwd.argtypes = [vp, vp, vp, i64, i64, ci]
        lib.ln_softmax_fwd.restype = ci
        lib.ln_fwd_from_partials.argtypes = [vp, vp, vp, i64, i64, ci, vp, vp, f32, ci, ci, vp,
                                             vp, vp, vp, vp, i64, i64, ci]
        lib.ln_fwd_from_partials.restype = ci
        lib.ln_testing_select_kernels.argtypes = [ci, ci, ci]
        lib.ln_testing_select_kernels.restype = ci
        lib.ln_testing_plan.argtypes = [ci, i64, i64, ci, ci, ci, ctypes.POINTER(ci)]
        lib.ln_testing_plan.restype = ci
        lib.gn_fwd.argtypes = [vp, i64, i64, vp, vp, i64, f32, ci, ci, vp, i64, i64, vp, vp, vp,
                               i64, i64, i64, i64, ci, vp, sz]
        lib.gn_fwd.restype = ci
        lib.gn_bwd.argtypes = [vp, i64, i64, vp, i64, i64, vp, vp, i64, ci, ci, vp, vp, vp, i64,
                               i64, vp, vp, vp, i64, i64, i64, i64, ci, ci, vp, sz]
        lib.gn_bwd.restype = ci
        lib.gn_workspace_bytes.argtypes = [i64, i64, i64, i64, ci, ci, ctypes.POINTER(sz)]
        lib.gn_workspace_bytes.restype = ci
        lib.rope_fwd.argtypes = [vp, vp, vp, f32, ci, vp, i64, i64, i64, ci]
        lib.rope_fwd.restype = ci
        lib.rope_bwd.argtypes = [vp, vp, vp, f32, ci, vp, i64, i64, i64, ci, ci, vp, sz]
        lib.rope_bwd.restype = ci
        lib.rope_bwd_workspace_bytes.argtypes = [i64, ctypes.POINTER(sz)]
        lib.rope_bwd_workspace_bytes.restype = ci
        lib.rope_frequencies.argtypes = [i64, ctypes.c_double, ci, ctypes.c_double, i64,
                                         ctypes.c_double, ctypes.c_double, vp,
                                         ctypes.POINTER(f32)]
        lib.rope_frequencies.restype = ci
        lib.mx_matrix_bytes.argtypes = [ci, i64, i64, ctypes.POINTER(sz), ctypes.POINTER(sz)]
        lib.mx_matrix_bytes.restype = ci
        lib.mx_norm_fwd.argtypes = [vp, vp, vp, vp, vp, f32, ci, ci, vp, vp, vp, vp, vp, vp, ci]
        lib.mx_norm_fwd.restype = ci
        lib.mx_quantize.argtypes = [vp, i64, ci, vp, vp, ci]
        lib.mx_quantize.restype = ci
        lib.mx_dequantize.argtypes = [vp, vp, i64, vp, ci]
        lib.mx_dequantize.restype = ci
        lib.mx_product.argtypes = [vp, vp, f32, vp, vp, i64, vp, i64, vp, vp, vp, ci]
        lib.mx_product.restype = ci
        if os.path.isfile(marshal_path()):
            loader = importlib.machinery.ExtensionFileLoader("_marshal", marshal_path())
            spec = importlib.util.spec_from_loader("_marshal", loader)
            module = importlib.util.module_from_spec(spec)
            loader.exec_module(module)
            module.bind(*(ctypes.cast(f, vp).value for f in (
                lib.mx_matrix_bytes, lib.mx_norm_fwd, lib.mx_quantize, lib.mx_dequantize,
                lib.mx_product, lib.ln_fwd_from_partials)))
            _marshal = module
        _lib = lib
        return lib


def exported_symbols(prefix: str = "ln_") -> list[str]:
    """Names of the C entry points this binding wraps that start with
    ``prefix``: "ln_", "gn_" (group norm), "rope_" (rotary positions) or "mx_"
    (quantised matrices)."""
    names = ["ln_fwd", "ln_fwd_ex", "ln_bwd", "ln_bwd_ex", "ln_bwd_workspace_bytes",
             "ln_status_string", "ln_last_cuda_error", "ln_device_error", "ln_bwd_noalloc",
             "ln_softmax_fwd", "ln_testing_select_kernels", "ln_fwd_from_partials",
             "ln_testing_plan", "gn_fwd", "gn_bwd", "gn_workspace_bytes", "rope_fwd", "rope_bwd",
             "rope_bwd_workspace_bytes", "rope_frequencies", "mx_matrix_bytes", "mx_norm_fwd",
             "mx_quantize", "mx_dequantize", "mx_product"]
    return [n for n in names if n.startswith(prefix)]


_FAMILY_CODES = {"default": 0, "ring": 1}


def ln_testing_select_kernels(forward="default", backward="default", softmax="default") -> None:
    """Testing hook (include/normfuse_testing.h): plan later calls with the
    default kernels of each shape ("default") or with the bulk-copy ring
    kernels ("ring"), per direction. Process-wide."""
    lib = load_library()
    try:
        codes = [_FAMILY_CODES[v] for v in (forward, backward, softmax)]
    except KeyError as e:
        raise ValueError(f"unknown kernel family {e.args[0]!r}") from None
    st = lib.ln_testing_select_kernels(*codes)
    if st:
        raise NormError(st, "ln_testing_select_kernels")


_PLAN_DIRECTIONS = {"forward": 0, "backward": 1, "softmax": 2, "partials": 3}
_PLAN_FIELDS = ("kind", "group", "n", "block", "grid", "smem")


def ln_testing_plan(direction, rows, hidden, dtype, mode="layernorm", option=False) -> dict:
    """Testing hook (include/normfuse_testing.h): the launch the library
    would plan for this shape on the current device, as a dict of kind,
    group, n, block, grid and smem. ``direction`` is "forward", "backward",
    "softmax" or "partials"; ``option`` a residual (forward) or dbias
    (backward)."""
    lib = load_library()
    try:
        d = _PLAN_DIRECTIONS[direction]
    except KeyError:
        raise ValueError(f"unknown direction {direction!r}") from None
    code = _DTYPE_CODES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    out = (ctypes.c_int * 6)()
    st = lib.ln_testing_plan(d, int(rows), int(hidden), code, _mode(mode), int(bool(option)), out)
    if st:
        raise NormError(st, "ln_testing_plan")
    return dict(zip(_PLAN_FIELDS, list(out)))


def ln_status_string(status: int) -> str:
    return load_library().ln_status_string(int(status)).decode()


def ln_last_cuda_error() -> int:
    return int(load_library().ln_last_cuda_error())


def ln_device_error(stream=None) -> int:
    """Wait for ``stream`` and return (and clear) the kernels' device error
    bits; 0 means no kernel reported a failed wait."""
    lib = load_library()
    flags = ctypes.c_uint(0)
    st = lib.ln_device_error(_stream(stream), ctypes.byref(flags))
    if st:
        raise NormError(st, "ln_device_error")
    return int(flags.value)


def _ptr(t) -> int | None:
    if t is None:
        return None
    try:
        address, here = t.data_ptr(), t.is_cuda
    except AttributeError:
        raise TypeError(f"expected a torch.Tensor or None, got {type(t).__name__}") from None
    if not here and t.numel():
        raise ValueError("tensors passed to the CUDA library must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return address or None


def _stream(stream) -> int | None:
    if stream is None:
        return _raw_stream(_get_device()) or None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream or None
    return int(stream) or None


def _shape(t: torch.Tensor) -> tuple[int, int]:
    if t.dim() < 1:
        raise ValueError("expected at least one dimension (the hidden one)")
    hidden = t.shape[-1]
    return t.numel() // hidden if hidden else 0, hidden


def _mode(mode) -> int:
    try:
        return _MODE_CODES[mode]
    except KeyError:
        raise ValueError(f"unknown mode {mode!r}") from None


def _dtype(t: torch.Tensor) -> int:
    try:
        return _DTYPE_CODES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def ln_fwd(x, bias, residual, gamma, beta, eps, mode, zero_centered_gamma, out_sum, y,
           mean, rstd, amax, stream=None) -> None:
    """Enqueue the fused forward on ``stream`` (default: torch's current stream).

    Tensors: x, residual, out_sum, y are [..., hidden] in one dtype; bias, gamma,
    beta are [hidden]; mean, rstd fp32 [rows]; amax a one-element fp32 tensor.
    Optional ones may be None (see ``ln_fwd`` in include/normfuse.h).
    """
    lib = load_library()
    rows, hidden = _shape(x)
    st = lib.ln_fwd(_ptr(x), _ptr(bias), _ptr(residual), _ptr(gamma), _ptr(beta),
                    float(eps), _mode(mode), int(bool(zero_centered_gamma)), _ptr(out_sum),
                    _ptr(y), _ptr(mean), _ptr(rstd), _ptr(amax), _stream(stream), rows,
                    hidden, _dtype(x))
    if st:
        raise NormError(st, "ln_fwd")


def ln_fwd_ex(x, bias, residual, gamma, beta, eps, mode, zero_centered_gamma, out_sum, y,
              mean, rstd, amax, y_fp8, fp8_scale, stream=None) -> None:
    """``ln_fwd`` plus an FP8 E4M3 copy of y: ``y_fp8`` is a uint8 (or
    torch.float8_e4m3fn) tensor shaped like x, ``fp8_scale`` a one-element fp32
    CUDA tensor; y may be None when y_fp8 is given."""
    lib = load_library()
    rows, hidden = _shape(x)
    st = lib.ln_fwd_ex(_ptr(x), _ptr(bias), _ptr(residual), _ptr(gamma), _ptr(beta),
                       float(eps), _mode(mode), int(bool(zero_centered_gamma)), _ptr(out_sum),
                       _ptr(y), _ptr(mean), _ptr(rstd), _ptr(amax), _ptr(y_fp8),
                       _ptr(fp8_scale), _stream(stream), rows, hidden, _dtype(x))
    if st:
        raise NormError(st, "ln_fwd_ex")


def _partials(kind) -> int:
    try:
        return _PARTIAL_CODES[kind]
    except KeyError:
        raise ValueError(f"unknown partial kind {kind!r}") from None


def ln_fwd_from_partials(x, psum, psq, tile_cols, kind, gamma, beta, eps, mode,
                         zero_centered_gamma, y, mean, rstd, amax, stream=None) -> None:
    """Enqueue the normalize step with row statistics combined from per
    column-tile partials: ``psum``/``psq`` are fp32 [rows, ceil(hidden /
    tile_cols)] tensors, ``kind`` "sum_sq" or "sum_m2" (see
    ``ln_fwd_from_partials`` in include/normfuse.h)."""
    lib = load_library()
    rows, hidden = _shape(x)
    n_tiles = psum.shape[-1] if psum is not None else -(-hidden // int(tile_cols))
    st = lib.ln_fwd_from_partials(_ptr(x), _ptr(psum), _ptr(psq), int(n_tiles), int(tile_cols),
                                  _partials(kind), _ptr(gamma), _ptr(beta), float(eps), _mode(mode),
                                  int(bool(zero_centered_gamma)), _ptr(y), _ptr(mean),
                                  _ptr(rstd), _ptr(amax), _stream(stream), rows, hidden,
                                  _dtype(x))
    if st:
        raise NormError(st, "ln_fwd_from_partials")


def ln_bwd_workspace_bytes(rows: int, hidden: int, dtype, mode) -> int:
    lib = load_library()
    out = ctypes.c_size_t(0)
    code = _DTYPE_CODES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    st = lib.ln_bwd_workspace_bytes(int(rows), int(hidden), code, _mode(mode), ctypes.byref(out))
    if st:
        raise NormError(st, "ln_bwd_workspace_bytes")
    return int(out.value)


def ln_bwd(dy, x_sum, gamma, mean, rstd, dx, dgamma, dbeta, stream=None, *, mode="layernorm",
           zero_centered_gamma=False, workspace=None) -> None:
    """Enqueue the fused backward on ``stream``.

    ``workspace`` is a CUDA tensor of at least ``ln_bwd_workspace_bytes`` bytes;
    when None a fresh one is allocated through torch for this call.
    """
    lib = load_library()
    rows, hidden = _shape(dy)
    if workspace is None and rows > 0:
        need = ln_bwd_workspace_bytes(rows, hidden, dy.dtype, mode)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dy.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.ln_bwd(_ptr(dy), _ptr(x_sum), _ptr(gamma), _ptr(mean), _ptr(rstd), _ptr(dx),
                    _ptr(dgamma), _ptr(dbeta), _stream(stream), rows, hidden, _dtype(dy),
                    _mode(mode), int(bool(zero_centered_gamma)), _ptr(workspace), ws_bytes)
    if st:
        raise NormError(st, "ln_bwd")


def ln_bwd_noalloc(dy, x_sum, gamma, mean, rstd, dx, dgamma, dbeta, stream=None, *,
                   mode="layernorm", zero_centered_gamma=False) -> None:
    """``ln_bwd`` without a workspace: the library's static scratch array holds
    the partials, so neither this call nor the library allocates memory.

    For callers that cannot allocate device memory around the backward
    (see ``ln_bwd_noalloc`` in include/normfuse.h for the size limit and the
    rule that calls overlapping on the GPU race on the shared array).
    """
    lib = load_library()
    rows, hidden = _shape(dy)
    st = lib.ln_bwd_noalloc(_ptr(dy), _ptr(x_sum), _ptr(gamma), _ptr(mean), _ptr(rstd),
                            _ptr(dx), _ptr(dgamma), _ptr(dbeta), _stream(stream), rows, hidden,
                            _dtype(dy), _mode(mode), int(bool(zero_centered_gamma)))
    if st:
        raise NormError(st, "ln_bwd_noalloc")


def ln_bwd_ex(dy, x_sum, gamma, mean, rstd, dx, dgamma, dbeta, dbias, stream=None, *,
              mode="layernorm", zero_centered_gamma=False, workspace=None) -> None:
    """``ln_bwd`` that also writes ``dbias`` ([hidden], the column sum of dx:
    the gradient of the forward's bias; may be None). dgamma, dbeta and dbias
    share one dtype, float32, bfloat16 or float16, taken from ``dgamma``: the
    column totals are rounded once to it."""
    lib = load_library()
    rows, hidden = _shape(dy)
    if workspace is None and rows > 0:
        need = ln_bwd_workspace_bytes(rows, hidden, dy.dtype, mode)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dy.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.ln_bwd_ex(_ptr(dy), _ptr(x_sum), _ptr(gamma), _ptr(mean), _ptr(rstd), _ptr(dx),
                       _ptr(dgamma), _ptr(dbeta), _ptr(dbias), _stream(stream), rows, hidden,
                       _dtype(dy), _mode(mode), int(bool(zero_centered_gamma)),
                       _ptr(workspace), ws_bytes, _dtype(dgamma))
    if st:
        raise NormError(st, "ln_bwd_ex")


def ln_softmax_fwd(x, y, stream=None) -> None:
    """Enqueue the softmax over the last dimension of the contiguous CUDA
    tensor ``x`` into ``y`` (same shape and dtype; ``y`` may be ``x`` itself)."""
    lib = load_library()
    rows, hidden = _shape(x)
    if y is not x and (y.shape != x.shape or y.dtype != x.dtype):
        raise ValueError("y must have the shape and dtype of x")
    st = lib.ln_softmax_fwd(_ptr(x), _ptr(y), _stream(stream), rows, hidden, _dtype(x))
    if st:
        raise NormError(st, "ln_softmax_fwd")


def softmax_fwd(x, *, out=None, stream=None):
    """Softmax over the last dimension of a contiguous tensor; returns ``y``
    (allocated with torch unless ``out`` is given)."""
    y = torch.empty_like(x) if out is None else out
    ln_softmax_fwd(x, y, stream)
    return y


class Workspace:
    """A reusable workspace, grown on demand (allocated through torch). Calls
    that may run at the same time, replays of captured graphs among them, need
    one each. A buffer that it has outgrown is kept, as a graph captured with
    it writes there at every replay; each buffer is at least twice the one
    before, so that what is kept is less than the newest one. ``release`` lets
    go of it."""

    def __init__(self, device=None):
        self.device = torch.device(device or "cuda")
        self.buf = torch.empty(0, dtype=torch.uint8, device=self.device)
        self.outgrown = []

    def get(self, rows: int, hidden: int, dtype, mode) -> torch.Tensor:
        return self.take(ln_bwd_workspace_bytes(rows, hidden, dtype, mode))

    def take(self, need: int) -> torch.Tensor:
        """A buffer of at least ``need`` bytes."""
        have = self.buf.numel()
        if have < need:
            if have:
                self.outgrown.append(self.buf)
            self.buf = torch.empty(max(need, 2 * have), dtype=torch.uint8, device=self.device)
        return self.buf

    def release(self) -> None:
        """Let go of the buffers that it has outgrown: for when no graph
        captured with one of them will be replayed again and no call that was
        given one is still running."""
        self.outgrown.clear()


def fused_norm_fwd(x, gamma, beta=None, *, bias=None, residual=None, eps=1e-5,
                   mode="layernorm", zero_centered_gamma=False, store_sum=None, amax=False,
                   stream=None):
    """Allocate the outputs with torch and run ``ln_fwd``.

    Returns a dict with ``y``, ``sum`` (or None), ``mean`` (LayerNorm), ``rstd``,
    ``amax`` (or None).
    """
    rows, hidden = _shape(x)
    if store_sum is None:
        store_sum = bias is not None or residual is not None
    rms = _mode(mode) == LN_RMSNORM
    y = torch.empty_like(x)
    out_sum = torch.empty_like(x) if store_sum else None
    mean = None if rms else torch.empty(rows, dtype=torch.float32, device=x.device)
    rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    am = torch.empty(1, dtype=torch.float32, device=x.device) if amax else None
    ln_fwd(x, bias, residual, gamma, None if rms else beta, eps, mode, zero_centered_gamma,
           out_sum, y, mean, rstd, am, stream)
    return {"y": y, "sum": out_sum, "mean": mean, "rstd": rstd, "amax": am}


def fused_norm_fwd_from_partials(x, psum, psq, tile_cols, gamma, beta=None, *, kind="sum_sq",
                                 eps=1e-5, mode="layernorm", zero_centered_gamma=False,
                                 amax=False, stream=None):
    """Allocate the outputs with torch and run ``ln_fwd_from_partials``;
    returns a dict with ``y``, ``mean`` (LayerNorm), ``rstd``, ``amax``."""
    if stream is None and not amax and (_lib or load_library()) and _marshal:
        r = _marshal.norm_from_partials(x, psum, psq, tile_cols, _partials(kind), gamma, beta, eps,
                                        _mode(mode), zero_centered_gamma)
        if r is not None:
            y, mean, rstd = _made(r, "ln_fwd_from_partials")
            return {"y": y, "mean": mean, "rstd": rstd, "amax": None}
    rows, hidden = _shape(x)
    rms = _mode(mode) == LN_RMSNORM
    y = torch.empty_like(x)
    mean = None if rms else torch.empty(rows, dtype=torch.float32, device=x.device)
    rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    am = torch.empty(1, dtype=torch.float32, device=x.device) if amax else None
    ln_fwd_from_partials(x, psum, psq, tile_cols, kind, gamma, None if rms else beta, eps, mode,
                         zero_centered_gamma, y, mean, rstd, am, stream)
    return {"y": y, "mean": mean, "rstd": rstd, "amax": am}


def fused_norm_bwd(dy, x_sum, gamma, mean, rstd, *, mode="layernorm", zero_centered_gamma=False,
                   need_dbeta=True, need_dbias=False, grad_dtype=torch.float32,
                   workspace: Workspace | None = None, stream=None):
    """Allocate the outputs with torch and run ``ln_bwd`` (``ln_bwd_ex`` when
    ``need_dbias`` or a ``grad_dtype`` other than float32); returns dx,
    dgamma, dbeta, dbias."""
    rows, hidden = _shape(dy)
    rms = _mode(mode) == LN_RMSNORM
    dx = torch.empty_like(dy)
    g = dict(dtype=grad_dtype, device=dy.device)
    dgamma = torch.empty(hidden, **g)
    dbeta = torch.empty(hidden, **g) if (need_dbeta and not rms) else None
    dbias = torch.empty(hidden, **g) if need_dbias else None
    ws = workspace.get(rows, hidden, dy.dtype, mode) if workspace is not None else None
    if need_dbias or grad_dtype != torch.float32:
        ln_bwd_ex(dy, x_sum, gamma, mean, rstd, dx, dgamma, dbeta, dbias, stream, mode=mode,
                  zero_centered_gamma=zero_centered_gamma, workspace=ws)
    else:
        ln_bwd(dy, x_sum, gamma, mean, rstd, dx, dgamma, dbeta, stream, mode=mode,
               zero_centered_gamma=zero_centered_gamma, workspace=ws)
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta, "dbias": dbias}


# ---- group norm and rotary positions ------------------------------------------
# These take tensors of any strides (the last dimension contiguous), run on the
# device of their first tensor whatever the current one is, and allocate on the
# stream that they launch on, so that a buffer of theirs is not handed out again
# while the launch is using it.

def _device_of(where: str, first, *others) -> int:
    """Number of the CUDA device that all given tensors live on."""
    try:
        device = first.get_device()
        for t in others:
            if t is not None and t.get_device() != device:
                raise ValueError(f"{where}: tensors on {first.device} and {t.device}")
    except AttributeError:
        for t in (first, *others):
            if t is not None and not isinstance(t, torch.Tensor):
                raise TypeError(f"{where}: expected a torch.Tensor or None, got "
                                f"{type(t).__name__}") from None
        raise
    if device < 0:
        raise ValueError(f"{where}: tensors passed to the CUDA library must live on a CUDA device")
    return device


# torch's own fast paths to the current device and the raw current stream of a
# device, where it has them: the public calls take a few microseconds each.
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
               or (lambda device: torch.cuda.current_stream(device).cuda_stream))


def _elsewhere(device: int, stream) -> bool:
    """Whether a call has to make its device or stream current first."""
    return stream is not None or device != _get_device()


@contextlib.contextmanager
def _current(device: int, stream):
    """Make ``device`` and ``stream`` (a torch stream, a raw one or None)
    current, so that what the call allocates belongs to the stream that it
    launches on."""
    with torch.cuda.device(device):
        if stream is None:
            yield
            return
        if not isinstance(stream, torch.cuda.Stream):
            # 0 is the legacy default stream, torch's own default
            stream = (torch.cuda.ExternalStream(int(stream)) if int(stream)
                      else torch.cuda.default_stream())
        if stream.device.index != device:
            raise ValueError(f"stream of {stream.device} for tensors on cuda:{device}")
        with torch.cuda.stream(stream):
            yield


def _dense_last(t, name):
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")


def _rows_of(t, name):
    """(samples, rows, channels, sample stride, row stride) of [N, ..., C]."""
    shape, stride = t.shape, t.stride()
    if len(shape) < 2:
        raise ValueError(f"{name}: expected [samples, ..., channels]")
    if stride[-1] != 1:
        _dense_last(t, name)
    if len(shape) == 3:
        return shape[0], shape[1], shape[2], stride[0], stride[1] if shape[1] > 1 else 0
    rows, row = 1, 0
    for n, s in zip(shape[-2:0:-1], stride[-2:0:-1]):
        if n == 1:
            continue
        if rows > 1 and s != row * rows and rows * n > 0:
            raise ValueError(f"{name}: the dimensions between samples and channels must have one "
                             "stride from row to row")
        row = s if rows == 1 else row
        rows *= n
    return shape[0], rows, shape[-1], stride[0], row


def _affine(p, name, N, C, dtype):
    """Stride between samples of gamma or beta: 0 for [C], else that of [N, C]."""
    if p.dtype != dtype:
        raise TypeError(f"{name}: {p.dtype} with activations of {dtype}")
    _dense_last(p, name)
    if p.shape == (C,):
        return 0
    if p.shape == (N, C):
        return p.stride(0) if N > 1 else C
    raise ValueError(f"{name}: expected [{C}] or [{N}, {C}], got {list(p.shape)}")


def _affines(where, gamma, beta, N, C, dtype, grads=False):
    """gamma, beta and their stride between samples (0: shared). Parameters of
    each sample that are one row expanded over the samples work as shared ones;
    with ``grads`` each sample has a gradient of its own, so they are laid out,
    as are two whose strides differ."""
    given = [p for p in (gamma, beta) if p is not None]
    steps = {_affine(p, f"{where}: {n}", N, C, dtype)
             for p, n in ((gamma, "gamma"), (beta, "beta")) if p is not None}
    each = [p.dim() == 2 for p in given]
    if len(steps) > 1 or (grads and N > 1 and 0 in steps and any(each)):
        if not all(each):
            raise ValueError(f"{where}: gamma and beta must both be shared or both per sample")
        gamma, beta = (None if p is None else p.contiguous() for p in (gamma, beta))
        steps = {C}
    return gamma, beta, steps.pop() if steps else 0


def _activation(act) -> int:
    try:
        return _ACT_CODES[act]
    except KeyError:
        raise ValueError(f"unknown activation {act!r}") from None


def _same(where, name, t, ref):
    if t.shape != ref.shape or t.dtype != ref.dtype:
        raise ValueError(f"{where}: {name} must have the shape and dtype of x")


def _check_stats(where, mean, rstd, N, G, optional):
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if t is None and optional:
            continue
        if t is None or t.shape != (N, G) or t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be a contiguous float32 [{N}, {G}]")


def gn_workspace_bytes(samples, rows, channels, groups, dtype, backward=False) -> int:
    """Bytes of workspace ``gn_fwd`` or ``gn_bwd`` needs for this shape."""
    lib = load_library()
    out = ctypes.c_size_t(0)
    code = _DTYPE_CODES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    st = lib.gn_workspace_bytes(int(samples), int(rows), int(channels), int(groups), code,
                                int(bool(backward)), ctypes.byref(out))
    if st:
        raise NormError(st, "gn_workspace_bytes")
    return int(out.value)


# The answer depends on the shape and the device alone.
@functools.lru_cache(maxsize=4096)
def _gn_need(device, samples, rows, channels, groups, dtype, backward):
    return gn_workspace_bytes(samples, rows, channels, groups, dtype, backward)


@functools.lru_cache(maxsize=4096)
def _rope_need(device, head_dim):
    return rope_bwd_workspace_bytes(head_dim)


def _workspace(workspace, need, device):
    """(tensor to hold on to, address, bytes) of a call's workspace of `need`
    bytes: the caller's, or one for this call."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), need
    if isinstance(workspace, Workspace):
        workspace = workspace.take(need)
    if not workspace.numel():
        return None, None, 0
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be a contiguous tensor on cuda:{device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def gn_fwd(x, groups, gamma, beta, eps, activation, zero_centered_gamma, y, mean, rstd,
           stream=None, *, workspace=None) -> None:
    """Enqueue the group norm of ``x`` [samples, ..., channels] into ``y``.

    gamma and beta are [channels], [samples, channels] or None; mean and rstd
    fp32 [samples, groups] or None; ``activation`` "none", "silu" or "gelu";
    ``workspace`` a CUDA tensor of ``gn_workspace_bytes`` bytes or a
    ``Workspace`` (one is allocated for the call when None). See ``gn_fwd`` in
    include/normfuse.h.
    """
    device = _device_of("gn_fwd", x, gamma, beta, y, mean, rstd)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return gn_fwd(x, groups, gamma, beta, eps, activation, zero_centered_gamma, y, mean,
                          rstd, workspace=workspace)
    _gn_fwd(device, x, groups, gamma, beta, eps, activation, zero_centered_gamma, y, mean, rstd,
            workspace)


def _gn_fwd(device, x, groups, gamma, beta, eps, activation, zero_centered_gamma, y, mean, rstd,
            workspace):
    lib = _lib or load_library()
    dt = _dtype(x)
    N, R, C, xs, xr = _rows_of(x, "gn_fwd: x")
    _same("gn_fwd", "y", y, x)
    _, _, _, ys, yr = _rows_of(y, "gn_fwd: y")
    gamma, beta, ps = _affines("gn_fwd", gamma, beta, N, C, x.dtype)
    _check_stats("gn_fwd", mean, rstd, N, groups, True)
    held, ws, ws_bytes = _workspace(workspace, _gn_need(device, N, R, C, groups, dt, False), device)
    st = lib.gn_fwd(x.data_ptr() or None, xs, xr, None if gamma is None else gamma.data_ptr(),
                    None if beta is None else beta.data_ptr(), ps, eps, _activation(activation),
                    1 if zero_centered_gamma else 0, y.data_ptr() or None, ys, yr,
                    None if mean is None else mean.data_ptr(),
                    None if rstd is None else rstd.data_ptr(), _raw_stream(device) or None, N, R,
                    C, groups, dt,
                    ws, ws_bytes)
    if st:
        raise NormError(st, "gn_fwd")


def gn_bwd(dy, x, groups, gamma, beta, activation, zero_centered_gamma, mean, rstd, dx, dgamma,
           dbeta, stream=None, *, workspace=None) -> None:
    """Enqueue the backward of ``gn_fwd``: dx, and dgamma and dbeta (contiguous,
    the shape of gamma, one dtype of float32, bfloat16 or float16; may be
    None). See ``gn_bwd`` in include/normfuse.h."""
    device = _device_of("gn_bwd", x, dy, gamma, beta, mean, rstd, dx, dgamma, dbeta)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return gn_bwd(dy, x, groups, gamma, beta, activation, zero_centered_gamma, mean, rstd,
                          dx, dgamma, dbeta, workspace=workspace)
    _gn_bwd(device, dy, x, groups, gamma, beta, activation, zero_centered_gamma, mean, rstd, dx,
            dgamma, dbeta, workspace)


def _gn_bwd(device, dy, x, groups, gamma, beta, activation, zero_centered_gamma, mean, rstd, dx,
            dgamma, dbeta, workspace):
    lib = _lib or load_library()
    dt = _dtype(x)
    N, R, C, xs, xr = _rows_of(x, "gn_bwd: x")
    _same("gn_bwd", "dy", dy, x)
    _same("gn_bwd", "dx", dx, x)
    _, _, _, ds, dr = _rows_of(dy, "gn_bwd: dy")
    _, _, _, os_, or_ = _rows_of(dx, "gn_bwd: dx")
    gamma, beta, ps = _affines("gn_bwd", gamma, beta, N, C, x.dtype, grads=True)
    _check_stats("gn_bwd", mean, rstd, N, groups, False)
    grads = [g for g in (dgamma, dbeta) if g is not None]
    for g in grads:
        if (g.shape != ((N, C) if ps else (C,)) or not g.is_contiguous()
                or g.dtype != grads[0].dtype):
            raise ValueError("gn_bwd: dgamma and dbeta must be contiguous, of the shape of gamma "
                             "and of one dtype")
    held, ws, ws_bytes = _workspace(workspace, _gn_need(device, N, R, C, groups, dt, True), device)
    st = lib.gn_bwd(dy.data_ptr() or None, ds, dr, x.data_ptr() or None, xs, xr,
                    None if gamma is None else gamma.data_ptr(),
                    None if beta is None else beta.data_ptr(), ps, _activation(activation),
                    1 if zero_centered_gamma else 0, mean.data_ptr() or None,
                    rstd.data_ptr() or None, dx.data_ptr() or None, os_, or_,
                    None if dgamma is None else dgamma.data_ptr(),
                    None if dbeta is None else dbeta.data_ptr(), _raw_stream(device) or None, N, R,
                    C, groups, dt, _dtype(grads[0]) if grads else LN_F32, ws, ws_bytes)
    if st:
        raise NormError(st, "gn_bwd")


def fused_group_norm_fwd(x, groups, gamma=None, beta=None, *, eps=1e-5, activation="none",
                         zero_centered_gamma=False, out=None, workspace=None, stream=None):
    """Group norm of a channels-last tensor [samples, ..., channels] with an
    activation ("none", "silu", "gelu") behind it; returns a dict with ``y``,
    ``mean`` and ``rstd`` ([samples, groups], for the backward). An NCHW tensor
    in torch's channels_last format goes in as ``x.permute(0, 2, 3, 1)``.

    gamma and beta are [channels], or [samples, channels] for a scale and
    shift of each sample. ``x`` and ``out`` may be slices of the channels of
    wider tensors.
    """
    device = _device_of("fused_group_norm_fwd", x, gamma, beta, out)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return fused_group_norm_fwd(x, groups, gamma, beta, eps=eps, activation=activation,
                                        zero_centered_gamma=zero_centered_gamma, out=out,
                                        workspace=workspace)
    y = torch.empty_like(x) if out is None else out
    mean = torch.empty((x.shape[0], groups), dtype=torch.float32, device=device)
    rstd = torch.empty_like(mean)
    _gn_fwd(device, x, groups, gamma, beta, eps, activation, zero_centered_gamma, y, mean, rstd,
            workspace)
    return {"y": y, "mean": mean, "rstd": rstd}


def fused_group_norm_bwd(dy, x, groups, gamma, beta, mean, rstd, *, activation="none",
                         zero_centered_gamma=False, grad_dtype=torch.float32, workspace=None,
                         stream=None):
    """The backward of ``fused_group_norm_fwd`` from its x and statistics;
    returns a dict with ``dx``, ``dgamma`` and ``dbeta`` (None where gamma or
    beta is None)."""
    device = _device_of("fused_group_norm_bwd", x, dy, gamma, beta, mean, rstd)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return fused_group_norm_bwd(dy, x, groups, gamma, beta, mean, rstd,
                                        activation=activation,
                                        zero_centered_gamma=zero_centered_gamma,
                                        grad_dtype=grad_dtype, workspace=workspace)
    dx = torch.empty_like(x)
    dgamma = None if gamma is None else torch.empty(gamma.shape, dtype=grad_dtype, device=device)
    dbeta = None if beta is None else torch.empty(beta.shape, dtype=grad_dtype, device=device)
    _gn_bwd(device, dy, x, groups, gamma, beta, activation, zero_centered_gamma, mean, rstd, dx,
            dgamma, dbeta, workspace)
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def rope_frequencies(rot, base=10000.0, *, scaling="none", factor=1.0, original=4096,
                     turns_fast=32.0, turns_slow=1.0, device="cuda"):
    """(frequencies, scale) of rotary positions: a float64 [rot / 2] tensor of
    radians a position on ``device``, and the scale of cos and sin.

    ``scaling`` stretches the context ``original`` by ``factor``: "linear",
    "ntk" or "yarn" (see ``rope_frequencies`` in include/normfuse.h).
    """
    lib = load_library()
    try:
        code = _SCALING_CODES[scaling]
    except KeyError:
        raise ValueError(f"unknown scaling {scaling!r}") from None
    host = torch.empty(max(int(rot), 0) // 2, dtype=torch.float64)
    scale = ctypes.c_float(0)
    st = lib.rope_frequencies(int(rot), base, code, factor, int(original), turns_fast, turns_slow,
                              host.data_ptr() or None, ctypes.byref(scale))
    if st:
        raise NormError(st, "rope_frequencies")
    return host.to(device), float(scale.value)


def rope_axes(*frequencies):
    """Frequencies for positions of several axes: the pairs of the first one
    turn with the first axis, those of the next with the next, and so on.
    Returns [axes, sum of the pairs]."""
    pairs = sum(f.numel() for f in frequencies)
    out = torch.zeros(len(frequencies), pairs, dtype=torch.float64, device=frequencies[0].device)
    at = 0
    for a, f in enumerate(frequencies):
        out[a, at:at + f.numel()] = f
        at += f.numel()
    return out


def _heads(t, name, like=None):
    """Shape [batch, tokens, heads, dim] and the strides of the first three, of
    [tokens, heads, dim] or [batch, tokens, heads, dim]."""
    shape, st = t.shape, t.stride()
    if like is not None and (shape != like.shape or t.dtype != like.dtype):
        raise ValueError(f"{name}: expected {list(like.shape)} of {like.dtype}")
    if st[-1:] != (1,):
        if len(shape) not in (3, 4):
            raise ValueError(f"{name}: expected [tokens, heads, dim] or "
                             "[batch, tokens, heads, dim]")
        _dense_last(t, name)
    if len(shape) == 4:
        return shape, st[:3]
    if len(shape) == 3:
        return (1, *shape), (0, *st[:2])
    raise ValueError(f"{name}: expected [tokens, heads, dim] or [batch, tokens, heads, dim]")


def _positions(where, positions, freqs, interleaved, scale, shape, dims):
    """The packed rope_positions struct."""
    if positions.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"{where}: positions must be int32 or int64, got {positions.dtype}")
    if freqs.dtype != torch.float64 or not freqs.is_contiguous() or freqs.dim() not in (1, 2):
        raise ValueError(f"{where}: frequencies must be a contiguous float64 [pairs] or "
                         "[axes, pairs]")
    axes = freqs.shape[0] if freqs.dim() == 2 else 1
    p, batch, tokens = positions, shape[0], shape[1]
    want, step = list(p.shape), list(p.stride())
    axis = 0
    if freqs.dim() == 2:
        if not want or want[0] != axes:
            raise ValueError(f"{where}: positions must start with the {axes} axes of the "
                             "frequencies")
        axis = step[0]
        want, step = want[1:], step[1:]
    if len(want) == 1 and want[0] == tokens:
        strides = (axis, 0, step[0])
    elif len(want) == 2 and want[0] == batch and want[1] == tokens and dims == 4:
        strides = (axis, step[0], step[1])
    else:
        raise ValueError(f"{where}: positions must be [tokens] or [batch, tokens] (behind the "
                         f"axes), got {list(p.shape)} for {batch} x {tokens}")
    return _ROPE_POSITIONS.pack(p.data_ptr(), 32 if p.dtype == torch.int32 else 64, axes, *strides,
                                freqs.data_ptr(), 2 * freqs.shape[-1], 1 if interleaved else 0,
                                scale)


def _gamma_ptr(g, name, D, dtype):
    if g is None:
        return 0
    if g.shape != (D,) or g.dtype != dtype or not g.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous [{D}] of {dtype}")
    return g.data_ptr()


def rope_fwd(q, k, positions, freqs, q_gamma, k_gamma, eps, zero_centered_gamma, interleaved,
             scale, out_q, out_k, stream=None) -> None:
    """Enqueue the rotary positions of ``q`` and ``k`` (k may be None), with the
    RMSNorm of each head where its gamma is given. Tensors are
    [batch, tokens, heads, dim] or [tokens, heads, dim] of any strides; an
    output may be its input. See ``rope_fwd`` in include/normfuse.h."""
    device = _device_of("rope_fwd", q, k, positions, freqs, q_gamma, k_gamma, out_q, out_k)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return rope_fwd(q, k, positions, freqs, q_gamma, k_gamma, eps, zero_centered_gamma,
                            interleaved, scale, out_q, out_k)
    _rope_fwd(device, q, k, positions, freqs, q_gamma, k_gamma, eps, zero_centered_gamma,
              interleaved, scale, out_q, out_k)


def _rope_fwd(device, q, k, positions, freqs, q_gamma, k_gamma, eps, zero_centered_gamma,
              interleaved, scale, out_q, out_k):
    lib = _lib or load_library()
    shape, xs = _heads(q, "rope_fwd: q")
    _, ys = _heads(out_q, "rope_fwd: out_q", q)
    D = shape[3]
    qs = _ROPE_HEADS.pack(q.data_ptr(), out_q.data_ptr(),
                          _gamma_ptr(q_gamma, "rope_fwd: q_gamma", D, q.dtype), shape[2], *xs, *ys)
    ks = None
    if (k is None) != (out_k is None):
        raise ValueError("rope_fwd: k and out_k go together")
    if k is not None:
        kshape, xs = _heads(k, "rope_fwd: k")
        _, ys = _heads(out_k, "rope_fwd: out_k", k)
        if kshape[:2] != shape[:2] or kshape[3] != D or k.dtype != q.dtype or k.dim() != q.dim():
            raise ValueError("rope_fwd: q and k must share batch, tokens, dim and dtype")
        ks = _ROPE_HEADS.pack(k.data_ptr(), out_k.data_ptr(),
                              _gamma_ptr(k_gamma, "rope_fwd: k_gamma", D, q.dtype), kshape[2], *xs,
                              *ys)
    pos = _positions("rope_fwd", positions, freqs, interleaved, scale, shape, q.dim())
    st = lib.rope_fwd(qs, ks, pos, eps, 1 if zero_centered_gamma else 0,
                      _raw_stream(device) or None, shape[0],
                      shape[1], D, _dtype(q))
    if st:
        raise NormError(st, "rope_fwd")


def rope_bwd_workspace_bytes(head_dim) -> int:
    """Bytes of workspace ``rope_bwd`` needs for the gradients of gammas."""
    lib = load_library()
    out = ctypes.c_size_t(0)
    st = lib.rope_bwd_workspace_bytes(int(head_dim), ctypes.byref(out))
    if st:
        raise NormError(st, "rope_bwd_workspace_bytes")
    return int(out.value)


def rope_bwd(dq, dk, q, k, positions, freqs, q_gamma, k_gamma, eps, zero_centered_gamma,
             interleaved, scale, out_dq, out_dk, dq_gamma, dk_gamma, stream=None, *,
             workspace=None) -> None:
    """Enqueue the backward of ``rope_fwd``: ``dq`` and ``dk`` are the gradients
    of its outputs, ``out_dq`` and ``out_dk`` those of its inputs (an output
    may be its gradient). q and k are needed with a gamma only; dq_gamma and
    dk_gamma ([dim], one dtype) may be None."""
    device = _device_of("rope_bwd", dq, dk, q, k, positions, freqs, q_gamma, k_gamma, out_dq,
                        out_dk, dq_gamma, dk_gamma)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return rope_bwd(dq, dk, q, k, positions, freqs, q_gamma, k_gamma, eps,
                            zero_centered_gamma, interleaved, scale, out_dq, out_dk, dq_gamma,
                            dk_gamma, workspace=workspace)
    _rope_bwd(device, dq, dk, q, k, positions, freqs, q_gamma, k_gamma, eps, zero_centered_gamma,
              interleaved, scale, out_dq, out_dk, dq_gamma, dk_gamma, workspace)


def _rope_bwd(device, dq, dk, q, k, positions, freqs, q_gamma, k_gamma, eps, zero_centered_gamma,
              interleaved, scale, out_dq, out_dk, dq_gamma, dk_gamma, workspace):
    lib = _lib or load_library()
    shape, _ = _heads(dq, "rope_bwd: dq")
    D = shape[3]
    if (dk is None) != (out_dk is None) or (dk is None and dk_gamma is not None):
        raise ValueError("rope_bwd: dk, out_dk and dk_gamma go together")
    grads = [g for g in (dq_gamma, dk_gamma) if g is not None]
    for g in grads:
        if g.shape != (D,) or not g.is_contiguous() or g.dtype != grads[0].dtype:
            raise ValueError(f"rope_bwd: dq_gamma and dk_gamma must be contiguous [{D}] of one "
                             "dtype")

    def side(d, x, gamma, out, dgamma, name):
        if d is None:
            return None
        dshape, ds = _heads(d, f"rope_bwd: d{name}")
        if (dshape[:2] != shape[:2] or dshape[3] != D or d.dtype != dq.dtype
                or d.dim() != dq.dim()):
            raise ValueError("rope_bwd: dq and dk must share batch, tokens, dim and dtype")
        _, os_ = _heads(out, f"rope_bwd: out_d{name}", d)
        xs = (0, 0, 0)
        if gamma is not None:
            if x is None:
                raise ValueError(f"rope_bwd: {name} is needed with its gamma")
            _, xs = _heads(x, f"rope_bwd: {name}", d)
        return _ROPE_HEADS_GRAD.pack(
            d.data_ptr(), 0 if gamma is None else x.data_ptr(), out.data_ptr(),
            _gamma_ptr(gamma, f"rope_bwd: {name}_gamma", D, d.dtype),
            0 if dgamma is None else dgamma.data_ptr(), dshape[2], *ds, *xs, *os_)

    qs = side(dq, q, q_gamma, out_dq, dq_gamma, "q")
    ks = side(dk, k, k_gamma, out_dk, dk_gamma, "k")
    pos = _positions("rope_bwd", positions, freqs, interleaved, scale, shape, dq.dim())
    held, ws, ws_bytes = _workspace(workspace, _rope_need(device, D) if grads else 0, device)
    st = lib.rope_bwd(qs, ks, pos, eps, 1 if zero_centered_gamma else 0,
                      _raw_stream(device) or None, shape[0],
                      shape[1], D, _dtype(dq), _dtype(grads[0]) if grads else LN_F32, ws, ws_bytes)
    if st:
        raise NormError(st, "rope_bwd")


def fused_rope_fwd(q, k, positions, freqs, *, q_gamma=None, k_gamma=None, eps=1e-6,
                   zero_centered_gamma=False, interleaved=False, scale=1.0, out_q=None, out_k=None,
                   stream=None):
    """Rotary positions of queries and keys [batch, tokens, heads, dim] (or
    [tokens, heads, dim]), with the RMSNorm of each head before the rotation
    where a gamma is given; returns a dict with ``q`` and ``k``.

    ``positions`` are int32 or int64 [tokens] or [batch, tokens]; ``freqs`` is
    what ``rope_frequencies`` gives ([pairs]: 2 * pairs elements of a head are
    rotated, the others pass through), or [axes, pairs] from ``rope_axes``
    with positions of [axes, ...]. ``out_q=q`` and ``out_k=k`` work in place.
    """
    device = _device_of("fused_rope_fwd", q, k, positions, freqs, q_gamma, k_gamma, out_q, out_k)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return fused_rope_fwd(q, k, positions, freqs, q_gamma=q_gamma, k_gamma=k_gamma,
                                  eps=eps, zero_centered_gamma=zero_centered_gamma,
                                  interleaved=interleaved, scale=scale, out_q=out_q, out_k=out_k)
    if out_q is None:
        out_q = torch.empty_like(q)
    if out_k is None and k is not None:
        out_k = torch.empty_like(k)
    _rope_fwd(device, q, k, positions, freqs, q_gamma, k_gamma, eps, zero_centered_gamma,
              interleaved, scale, out_q, out_k)
    return {"q": out_q, "k": out_k}


def fused_rope_bwd(dq, dk, positions, freqs, *, q=None, k=None, q_gamma=None, k_gamma=None,
                   eps=1e-6, zero_centered_gamma=False, interleaved=False, scale=1.0,
                   grad_dtype=torch.float32, workspace=None, stream=None):
    """The backward of ``fused_rope_fwd``; ``q`` and ``k`` are its inputs,
    needed with a gamma. Returns a dict with ``dq``, ``dk``, ``dq_gamma`` and
    ``dk_gamma`` (None where there is none)."""
    device = _device_of("fused_rope_bwd", dq, dk, positions, freqs, q, k, q_gamma, k_gamma)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return fused_rope_bwd(dq, dk, positions, freqs, q=q, k=k, q_gamma=q_gamma,
                                  k_gamma=k_gamma, eps=eps,
                                  zero_centered_gamma=zero_centered_gamma,
                                  interleaved=interleaved, scale=scale, grad_dtype=grad_dtype,
                                  workspace=workspace)
    out_dq = torch.empty_like(dq)
    out_dk = torch.empty_like(dk) if dk is not None else None
    D = dq.shape[-1]
    gq = torch.empty(D, dtype=grad_dtype, device=device) if q_gamma is not None else None
    gk = (torch.empty(D, dtype=grad_dtype, device=device)
          if k_gamma is not None and dk is not None else None)
    _rope_bwd(device, dq, dk, q, k, positions, freqs, q_gamma, k_gamma, eps, zero_centered_gamma,
              interleaved, scale, out_dq, out_dk, gq, gk, workspace)
    return {"dq": out_dq, "dk": out_dk, "dq_gamma": gq, "dk_gamma": gk}


# ---- quantised matrices ----------------------------------------------------------

class Quantized(NamedTuple):
    """A matrix in 8 or 4 bits with scales (``mx_matrix`` in include/normfuse.h).

    ``format`` is "fp8_row", "fp8_block", "mxfp8", "mxfp4" or "nvfp4". ``codes``
    [rows, columns] are float8_e4m3fn, of the 4-bit formats uint8 with two codes a
    byte; microscaled rows are padded to 32 columns. ``scales`` are float32 [rows]
    or [rows, blocks], of the microscaled formats [rows / 128, blocks / 4, 32, 4, 4]
    (rounded up) of float8_e8m0fnu or, for nvfp4, float8_e4m3fn. ``mul`` is the
    float32 that nvfp4's values were multiplied by (one element; None: 1).
    """

    codes: torch.Tensor
    scales: torch.Tensor
    format: str
    rows: int
    cols: int
    mul: torch.Tensor | None = None


def _made(r, where):
    """What a function of csrc/marshal.cc made, or the error that a status is."""
    if isinstance(r, int):
        raise NormError(r, where)
    return r


def _format(format) -> int:
    try:
        return _FORMAT_CODES[format]
    except (KeyError, TypeError):
        raise ValueError(f"unknown format {format!r}") from None


def mx_matrix_bytes(format, rows, cols) -> tuple[int, int]:
    """Bytes of a quantised matrix's codes and of its scales."""
    lib = load_library()
    codes, scales = ctypes.c_size_t(0), ctypes.c_size_t(0)
    st = lib.mx_matrix_bytes(_format(format), int(rows), int(cols), ctypes.byref(codes),
                             ctypes.byref(scales))
    if st:
        raise NormError(st, "mx_matrix_bytes")
    return int(codes.value), int(scales.value)


@functools.lru_cache(maxsize=4096)
def _quantized_layout(fmt, rows, cols):
    """(shape and type of the codes, of the scales, bytes of either)."""
    rows, cols = int(rows), int(cols)
    e4m3 = torch.float8_e4m3fn
    bytes_of = mx_matrix_bytes(fmt, rows, cols)
    if fmt in ("fp8_row", "fp8_block"):
        scales = (rows,) if fmt == "fp8_row" else (rows, -(-cols // 128))
        return (rows, cols), e4m3, scales, torch.float32, bytes_of
    pitch = bytes_of[0] // rows if rows else -(-cols // 32) * (32 if fmt == "mxfp8" else 16)
    blocks = -(-cols // (16 if fmt == "nvfp4" else 32))
    return ((rows, pitch), e4m3 if fmt == "mxfp8" else torch.uint8,
            (-(-rows // 128), -(-blocks // 4), 32, 4, 4),
            e4m3 if fmt == "nvfp4" else torch.float8_e8m0fnu, bytes_of)


def quantized_empty(rows, cols, format, *, mul=None, device="cuda") -> Quantized:
    """A matrix with room for codes and scales, not initialised."""
    cshape, ctype, sshape, stype, _ = _quantized_layout(format, rows, cols)
    return Quantized(torch.empty(cshape, dtype=ctype, device=device),
                     torch.empty(sshape, dtype=stype, device=device), format, rows, cols, mul)


def _matrix(where, q):
    """The packed mx_matrix struct of ``q``."""
    codes, scales, format, rows, cols, mul = q
    need = _quantized_layout(format, rows, cols)[4]
    if (codes.nbytes != need[0] or scales.nbytes != need[1] or not codes.is_contiguous()
            or not scales.is_contiguous()):
        raise ValueError(f"{where}: codes and scales of {rows} x {cols} {format} must be "
                         f"contiguous, of {need[0]} and {need[1]} bytes")
    if mul is None or format != "nvfp4":
        return _MX_MATRIX.pack(codes.data_ptr(), scales.data_ptr(), 0, _FORMAT_CODES[format], rows,
                               cols)
    if mul.numel() != 1 or mul.dtype != torch.float32:
        raise ValueError(f"{where}: mul must be one float32")
    return _MX_MATRIX.pack(codes.data_ptr(), scales.data_ptr(), mul.data_ptr(), MX_NVFP4, rows,
                           cols)


def mx_norm_fwd(x, bias, residual, gamma, beta, eps, mode, zero_centered_gamma, out_sum, y, mean,
                rstd, q, stream=None) -> None:
    """Enqueue the fused forward of ``ln_fwd`` with its result in ``q`` (a
    ``Quantized`` of [rows, hidden]); y may be None. See ``mx_norm_fwd`` in
    include/normfuse.h."""
    device = _device_of("mx_norm_fwd", x, bias, residual, gamma, beta, out_sum, y, mean, rstd,
                        q.codes, q.scales, q.mul)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return mx_norm_fwd(x, bias, residual, gamma, beta, eps, mode, zero_centered_gamma,
                               out_sum, y, mean, rstd, q)
    rows, hidden = _shape(x)
    if (q.rows, q.cols) != (rows, hidden):
        raise ValueError(f"mx_norm_fwd: q must be {rows} x {hidden}, is {q.rows} x {q.cols}")
    for n, t in (("out_sum", out_sum), ("y", y)):
        if t is not None and (t.shape != x.shape or t.dtype != x.dtype or not t.is_contiguous()):
            raise ValueError(f"mx_norm_fwd: {n} must be contiguous, of the shape and dtype of x")
    for n, t in (("mean", mean), ("rstd", rstd)):
        if t is not None and (t.shape != (rows,) or t.dtype != torch.float32
                              or not t.is_contiguous()):
            raise ValueError(f"mx_norm_fwd: {n} must be a contiguous float32 [{rows}]")
    _mx_norm_fwd(device, x, bias, residual, gamma, beta, eps, _mode(mode), zero_centered_gamma,
                 out_sum, y, mean, rstd, q)


def _mx_norm_fwd(device, x, bias, residual, gamma, beta, eps, mode, zero_centered_gamma, out_sum,
                 y, mean, rstd, q):
    """The call itself; outputs and q's shape are as they should be."""
    lib = _lib or load_library()
    dt = _dtype(x)
    if not x.is_contiguous():
        raise ValueError("mx_norm_fwd: x must be contiguous")
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype
                                 or not residual.is_contiguous()):
        raise ValueError("mx_norm_fwd: residual must be contiguous, of the shape and dtype of x")
    n = q.cols
    for name, t in (("gamma", gamma), ("beta", beta), ("bias", bias)):
        if t is not None and (t.numel() != n or t.dtype != x.dtype or not t.is_contiguous()):
            raise ValueError(f"mx_norm_fwd: {name} must be a contiguous [{n}] of {x.dtype}")
    st = lib.mx_norm_fwd(
        x.data_ptr() or None, None if bias is None else bias.data_ptr(),
        None if residual is None else residual.data_ptr() or None,
        None if gamma is None else gamma.data_ptr(), None if beta is None else beta.data_ptr(),
        eps, mode, 1 if zero_centered_gamma else 0,
        None if out_sum is None else out_sum.data_ptr() or None,
        None if y is None else y.data_ptr() or None,
        None if mean is None else mean.data_ptr() or None,
        None if rstd is None else rstd.data_ptr() or None, _matrix("mx_norm_fwd", q),
        _raw_stream(device) or None, dt)
    if st:
        raise NormError(st, "mx_norm_fwd")


def _plane(where, name, t, shape=None, dtype=None):
    """Row stride of a matrix [rows, cols] whose columns are contiguous."""
    size = t.shape
    if len(size) != 2 or (shape is not None and size != shape) or (dtype and t.dtype != dtype):
        raise ValueError(f"{where}: {name} must be "
                         + (f"{list(shape)} of {dtype}" if shape is not None else "a matrix"))
    row, col = t.stride()
    if col != 1 and size[1] > 1:
        raise ValueError(f"{where}: {name}: the last dimension must be contiguous")
    return row if size[0] > 1 else size[1]


def mx_quantize(x, q, *, transpose=False, stream=None) -> None:
    """Enqueue the quantisation of the matrix ``x`` (its transpose with
    ``transpose``) into ``q``; the rows of x may be any distance apart."""
    device = _device_of("mx_quantize", x, q.codes, q.scales, q.mul)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return mx_quantize(x, q, transpose=transpose)
    _mx_quantize(device, x, q, transpose)


def _mx_quantize(device, x, q, transpose):
    lib = _lib or load_library()
    row = _plane("mx_quantize", "x", x, (q.cols, q.rows) if transpose else (q.rows, q.cols), x.dtype)
    st = lib.mx_quantize(x.data_ptr() or None, row, 1 if transpose else 0,
                         _matrix("mx_quantize", q), _raw_stream(device) or None, _dtype(x))
    if st:
        raise NormError(st, "mx_quantize")


def mx_dequantize(q, y, stream=None) -> None:
    """Enqueue the values of ``q`` into the matrix ``y``."""
    device = _device_of("mx_dequantize", q.codes, q.scales, q.mul, y)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return mx_dequantize(q, y)
    _mx_dequantize(device, q, y)


def _mx_dequantize(device, q, y):
    lib = _lib or load_library()
    row = _plane("mx_dequantize", "y", y, (q.rows, q.cols), y.dtype)
    st = lib.mx_dequantize(_matrix("mx_dequantize", q), y.data_ptr() or None, row,
                           _raw_stream(device) or None, _dtype(y))
    if st:
        raise NormError(st, "mx_dequantize")


def mx_product(a, b, alpha, bias, residual, out, psum, psq, stream=None) -> None:
    """Enqueue out = alpha * a @ b.T + bias + residual of two microscaled
    matrices; psum and psq (float32 [rows, ceil(columns / 128)], or None) take
    the statistics of 128-column tiles for ``ln_fwd_from_partials``. See
    ``mx_product`` in include/normfuse.h."""
    device = _device_of("mx_product", out, a.codes, a.scales, a.mul, b.codes, b.scales, b.mul, bias,
                        residual, psum, psq)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return mx_product(a, b, alpha, bias, residual, out, psum, psq)
    _mx_product(device, a, b, alpha, bias, residual, out, psum, psq)


def _mx_product(device, a, b, alpha, bias, residual, out, psum, psq):
    lib = _lib or load_library()
    where, rows, cols, dtype = "mx_product", a.rows, b.rows, out.dtype
    shape = (rows, cols)
    row = _plane(where, "out", out, shape, dtype)
    res_row = row if residual is None else _plane(where, "residual", residual, shape, dtype)
    if bias is not None and (bias.numel() != cols or bias.dtype != dtype
                             or not bias.is_contiguous()):
        raise ValueError(f"{where}: bias must be a contiguous [{cols}] of {dtype}")
    for t in (psum, psq):
        if t is not None and (t.shape != (rows, -(-cols // 128)) or t.dtype != torch.float32
                              or not t.is_contiguous()):
            raise ValueError(f"{where}: psum and psq must be contiguous float32 "
                             f"[{rows}, {-(-cols // 128)}]")
    st = lib.mx_product(_matrix(where, a), _matrix(where, b), alpha,
                        None if bias is None else bias.data_ptr() or None,
                        None if residual is None else residual.data_ptr() or None, res_row,
                        out.data_ptr() or None, row,
                        None if psum is None else psum.data_ptr() or None,
                        None if psq is None else psq.data_ptr() or None,
                        _raw_stream(device) or None, _dtype(out))
    if st:
        raise NormError(st, where)


def fused_norm_quant_fwd(x, gamma, beta=None, *, format, mul=None, bias=None, residual=None,
                         eps=1e-5, mode="layernorm", zero_centered_gamma=False, store_sum=None,
                         store_y=False, stream=None):
    """The fused forward of ``fused_norm_fwd`` with its result quantised: returns
    a dict with ``q`` (a ``Quantized`` of [rows, hidden]), ``sum`` (or None),
    ``y`` (in x's dtype, with ``store_y``), ``mean`` (LayerNorm) and ``rstd``.

    ``fused_norm_bwd`` on ``sum`` (or x), ``mean`` and ``rstd`` is its backward,
    the gradient of the dequantised result passed straight through. ``mul`` is
    nvfp4's factor (one float32 on the device, commonly 2688 over the largest
    magnitude seen, which is the caller's to find).
    """
    if store_sum is None:
        store_sum = bias is not None or residual is not None
    if stream is None and (_lib or load_library()) and _marshal:
        r = _marshal.norm_quant(x, gamma, beta, bias, residual, mul, _format(format), _mode(mode),
                                zero_centered_gamma, eps, store_sum, store_y)
        if r is not None:
            codes, scales, out_sum, y, mean, rstd = _made(r, "mx_norm_fwd")
            return {"q": Quantized(codes, scales, format, codes.shape[0], x.shape[-1], mul),
                    "sum": out_sum, "y": y, "mean": mean, "rstd": rstd}
    device = _device_of("fused_norm_quant_fwd", x, gamma, beta, mul, bias, residual)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return fused_norm_quant_fwd(x, gamma, beta, format=format, mul=mul, bias=bias,
                                        residual=residual, eps=eps, mode=mode,
                                        zero_centered_gamma=zero_centered_gamma,
                                        store_sum=store_sum, store_y=store_y)
    rows, hidden = _shape(x)
    mode = _mode(mode)
    rms = mode == LN_RMSNORM
    q = quantized_empty(rows, hidden, format, mul=mul, device=device)
    out_sum = torch.empty_like(x) if store_sum else None
    y = torch.empty_like(x) if store_y else None
    mean = None if rms else torch.empty(rows, dtype=torch.float32, device=device)
    rstd = torch.empty(rows, dtype=torch.float32, device=device)
    _mx_norm_fwd(device, x, bias, residual, gamma, None if rms else beta, eps, mode,
                 zero_centered_gamma, out_sum, y, mean, rstd, q)
    return {"q": q, "sum": out_sum, "y": y, "mean": mean, "rstd": rstd}


def quantize(x, format, *, mul=None, transpose=False, stream=None) -> Quantized:
    """The matrix ``x``, or its transpose, in 8 or 4 bits with scales. Rows of x
    may be any distance apart (a slice of a wider tensor)."""
    if stream is None and (_lib or load_library()) and _marshal:
        r = _marshal.quantize(x, _format(format), transpose, mul)
        if r is not None:
            codes, scales = _made(r, "mx_quantize")
            return Quantized(codes, scales, format, codes.shape[0], x.shape[0 if transpose else 1],
                             mul)
    device = _device_of("quantize", x, mul)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return quantize(x, format, mul=mul, transpose=transpose)
    if x.dim() != 2:
        raise ValueError("quantize: x must be a matrix")
    rows, cols = x.shape[::-1] if transpose else x.shape
    q = quantized_empty(rows, cols, format, mul=mul, device=device)
    _mx_quantize(device, x, q, transpose)
    return q


def dequantize(q, dtype=torch.float32, *, out=None, stream=None):
    """The values of ``q`` as a [rows, cols] tensor of ``dtype``."""
    if stream is None and out is None and (_lib or load_library()) and _marshal:
        codes, scales, format, rows, cols, mul = q
        r = _marshal.dequantize(codes, scales, mul, _format(format), rows, cols,
                                _DTYPE_CODES.get(dtype, -1))
        if r is not None:
            return _made(r, "mx_dequantize")
    device = _device_of("dequantize", q.codes, q.scales, q.mul, out)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return dequantize(q, dtype, out=out)
    if out is None:
        out = torch.empty((q.rows, q.cols), dtype=dtype, device=device)
    _mx_dequantize(device, q, out)
    return out


def scaled_product(a, b, *, alpha=1.0, bias=None, residual=None, dtype=torch.bfloat16, out=None,
                   partials=False, stream=None):
    """alpha * a @ b.T + bias + residual of two ``Quantized`` matrices of one
    microscaled format with equal columns (activations and a projection's
    weights); returns a dict with ``out`` [a.rows, b.rows] and, with
    ``partials``, ``psum``, ``psq`` and ``tile_cols`` for
    ``fused_norm_fwd_from_partials(..., kind="sum_m2")``.

    ``bias`` [b.rows] and ``residual`` [a.rows, b.rows] are of the output's
    dtype; ``out`` may be the residual itself. Its gradients are products, too:
    quantise the output's gradient and the weights (transpose=True) for the
    input's, both operands transposed for the weights'.
    """
    if (stream is None and a.format == b.format and a.cols == b.cols and (_lib or load_library())
            and _marshal):
        r = _marshal.product(a.codes, a.scales, a.mul, b.codes, b.scales, b.mul, _format(a.format),
                             a.rows, b.rows, a.cols, alpha, bias, residual,
                             _DTYPE_CODES.get(dtype, -1), out, partials)
        if r is not None:
            out, psum, psq = _made(r, "mx_product")
            return {"out": out, "psum": psum, "psq": psq, "tile_cols": 128}
    device = _device_of("scaled_product", a.codes, a.scales, a.mul, b.codes, b.scales, b.mul, bias,
                        residual, out)
    if _elsewhere(device, stream):
        with _current(device, stream):
            return scaled_product(a, b, alpha=alpha, bias=bias, residual=residual, dtype=dtype,
                                  out=out, partials=partials)
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=dtype, device=device)
    psum = psq = None
    if partials:
        shape = (a.rows, -(-b.rows // 128))
        psum = torch.empty(shape, dtype=torch.float32, device=device)
        psq = torch.empty(shape, dtype=torch.float32, device=device)
    _mx_product(device, a, b, alpha, bias, residual, out, psum, psq)
    return {"out": out, "psum": psum, "psq": psq, "tile_cols": 128}
