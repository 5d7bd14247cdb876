"""Quantised matrices without a GPU: declared and exported entry points, the
layout's sizes, refusals on the host (no call below reaches the GPU) and the
binding's own checks."""

import ctypes
import os
import re
import struct

import pytest
import torch

import normalization_fwd_gb300 as nf
from oracle import mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, ALIGN, SHAPE, UNSUPPORTED, CUDA, WORKSPACE, INVALID, SCRATCH_LIMIT = range(9)
X, B, R, G, BE, S, Y, M, RS, C, SC, MU, C2, SC2, P1, P2 = (0x7f0000000000 + i * 0x100000000 for i in range(16))
BF16 = 1


@pytest.fixture(scope="module")
def lib():
    nf.build_library()
    return nf.load_library()


def test_declared_entry_points_are_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "normfuse.h")).read(),
                  flags=re.S)
    names = sorted(set(re.findall(r"^ln_status (mx_\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(nf.exported_symbols("mx_"))
    for n in names:
        assert hasattr(lib, n), n
    for name in ("MX_FP8_ROW", "MX_FP8_BLOCK", "MX_MXFP8", "MX_MXFP4", "MX_NVFP4"):
        assert re.search(rf"{name} = {getattr(nf, name)}\b", text), name


@pytest.mark.parametrize("fmt", mx.FORMATS)
@pytest.mark.parametrize("rows,cols", [(0, 1), (1, 1), (5, 100), (129, 1165), (128, 64), (1000, 8192)])
def test_sizes_are_the_layouts(lib, fmt, rows, cols):
    codes, scales = nf.mx_matrix_bytes(fmt, rows, cols)
    if fmt in ("fp8_row", "fp8_block"):
        assert codes == rows * cols
        assert scales == 4 * rows * (1 if fmt == "fp8_row" else -(-cols // 128))
    else:
        assert codes == rows * -(-cols // 32) * (32 if fmt == "mxfp8" else 16)
        assert scales == -(-rows // 128) * -(-(-(-cols // mx.BLOCK[fmt])) // 4) * 512
    q = nf.quantized_empty(rows, cols, fmt, device="cpu")
    assert (q.codes.nbytes, q.scales.nbytes) == (codes, scales)


def matrix(codes=C, scales=SC, mul=0, fmt=2, rows=40, cols=64):
    return struct.pack("@PPPiqq", codes or 0, scales or 0, mul or 0, fmt, rows, cols)


MATRIX_REFUSALS = [
    (dict(codes=None), NULL),
    (dict(scales=None), NULL),
    (dict(fmt=5), UNSUPPORTED),
    (dict(fmt=-1), UNSUPPORTED),
    (dict(rows=-1), SHAPE),
    (dict(cols=0), SHAPE),
    (dict(rows=(1 << 31) - 128), SHAPE),
    (dict(cols=1 << 31), SHAPE),
    (dict(codes=C + 8), ALIGN),
    (dict(scales=SC + 8), ALIGN),
    (dict(fmt=0, scales=SC + 2), ALIGN),
    (dict(fmt=4, mul=MU + 2), ALIGN),
    (dict(scales=C), INVALID),                      # codes and scales in one another
]


def norm(lib, x=X, bias=B, res=R, g=G, be=BE, eps=1e-5, mode=0, s=S, y=Y, m=M, r=RS, dt=BF16, q=None, **kw):
    return lib.mx_norm_fwd(x, bias, res, g, be, eps, mode, 0, s, y, m, r, matrix(**kw) if q is None else q,
                           None, dt)


@pytest.mark.parametrize("kw,want", MATRIX_REFUSALS + [
    (dict(x=None), NULL),
    (dict(g=None), NULL),
    (dict(dt=3), UNSUPPORTED),
    (dict(mode=2), UNSUPPORTED),
    (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(x=X + 1), ALIGN),
    (dict(m=M + 2), ALIGN),
    (dict(cols=16392), SHAPE),                      # wider than a row of 2048 vectors, or 8192 one by one
    (dict(cols=8193), SHAPE),
    (dict(y=X), INVALID),
    (dict(s=R + 64), INVALID),
    (dict(codes=X), INVALID),
    (dict(scales=Y), INVALID),
    (dict(fmt=4, mul=C + 16), INVALID),             # the factor within the codes
])
def test_norm_rejects_on_host(lib, kw, want):
    assert norm(lib, **kw) == want


def test_norm_without_a_matrix(lib):
    assert lib.mx_norm_fwd(X, None, None, G, None, 1e-5, 1, 0, None, None, None, RS, None, None, BF16) == NULL


def quantize(lib, x=X, row=64, t=0, dt=BF16, **kw):
    return lib.mx_quantize(x, row, t, matrix(**kw), None, dt)


@pytest.mark.parametrize("t", [0, 1])
@pytest.mark.parametrize("kw,want", MATRIX_REFUSALS + [
    (dict(x=None), NULL),
    (dict(dt=-1), UNSUPPORTED),
    (dict(row=-1), INVALID),
    (dict(row=1 << 60), INVALID),
    (dict(x=X + 1), ALIGN),
    (dict(codes=X + 64), INVALID),
    (dict(scales=X), INVALID),
    (dict(fmt=4, mul=SC), INVALID),
])
def test_quantize_rejects_on_host(lib, kw, want, t):
    assert quantize(lib, t=t, **kw) == want


def dequantize(lib, y=Y, row=64, dt=BF16, **kw):
    return lib.mx_dequantize(matrix(**kw), y, row, None, dt)


@pytest.mark.parametrize("kw,want", MATRIX_REFUSALS[:-1] + [
    (dict(y=None), NULL),
    (dict(dt=7), UNSUPPORTED),
    (dict(row=63), INVALID),
    (dict(y=Y + 1), ALIGN),
    (dict(y=C), INVALID),
    (dict(y=SC), INVALID),
    (dict(fmt=4, mul=Y + 4), INVALID),
])
def test_dequantize_rejects_on_host(lib, kw, want):
    assert dequantize(lib, **kw) == want


def product(lib, a={}, b={}, alpha=1.0, bias=None, res=None, res_row=50, out=Y, out_row=50, ps=None, pq=None, dt=BF16):
    return lib.mx_product(matrix(**a), matrix(**{**dict(codes=C2, scales=SC2, rows=50), **b}), alpha, bias, res,
                          res_row, out, out_row, ps, pq, None, dt)


@pytest.mark.parametrize("kw,want", [(dict(a=k), w) for k, w in MATRIX_REFUSALS[:-1] if "fmt" not in k and "cols" not in k]
                         + [(dict(b=k), w) for k, w in MATRIX_REFUSALS[:-1] if "fmt" not in k and "cols" not in k] + [
    (dict(a=dict(fmt=3)), UNSUPPORTED),             # two formats
    (dict(a=dict(fmt=0), b=dict(fmt=0)), UNSUPPORTED),   # not microscaled
    (dict(a=dict(fmt=1), b=dict(fmt=1)), UNSUPPORTED),
    (dict(a=dict(fmt=9), b=dict(fmt=9)), UNSUPPORTED),
    (dict(a=dict(cols=32)), SHAPE),                 # not as long as the other's rows
    (dict(a=dict(cols=0), b=dict(cols=0)), SHAPE),
    (dict(dt=3), UNSUPPORTED),
    (dict(alpha=float("inf")), INVALID),
    (dict(alpha=float("nan")), INVALID),
    (dict(out=None), NULL),
    (dict(ps=P1), NULL),                            # statistics go together
    (dict(pq=P1), NULL),
    (dict(out_row=49), INVALID),
    (dict(res=R, res_row=49), INVALID),
    (dict(out_row=1 << 60), INVALID),
    (dict(out=Y + 1), ALIGN),
    (dict(bias=B + 1), ALIGN),
    (dict(res=R + 1), ALIGN),
    (dict(ps=P1 + 2, pq=P2), ALIGN),
    (dict(out=C), INVALID),
    (dict(out=SC2), INVALID),
    (dict(out=B, bias=B + 64), INVALID),
    (dict(res=Y + 2), INVALID),                     # in place is the same pointer
    (dict(res=Y, res_row=64), INVALID),             # and the same rows
    (dict(ps=Y, pq=P2), INVALID),
    (dict(ps=P1, pq=P1), INVALID),
    (dict(a=dict(fmt=4, mul=Y), b=dict(fmt=4)), INVALID),
])
def test_product_rejects_on_host(lib, kw, want):
    assert product(lib, **kw) == want


def test_calls_without_rows_do_nothing(lib):
    """No rows: accepted without a device."""
    assert norm(lib, rows=0, x=None, codes=None, scales=None) == OK
    assert quantize(lib, rows=0, x=None, codes=None, scales=None) == OK
    assert dequantize(lib, rows=0, y=None, codes=None, scales=None) == OK
    assert product(lib, a=dict(rows=0, codes=None, scales=None), out=None) == OK
    assert product(lib, b=dict(rows=0, codes=None, scales=None), out=None, out_row=0, res_row=0) == OK


def test_null_outputs_of_sizes(lib):
    n = ctypes.c_size_t()
    assert lib.mx_matrix_bytes(2, 3, 4, None, ctypes.byref(n)) == NULL
    assert lib.mx_matrix_bytes(2, 3, 4, ctypes.byref(n), None) == NULL
    assert lib.mx_matrix_bytes(5, 3, 4, ctypes.byref(n), ctypes.byref(n)) == UNSUPPORTED
    assert lib.mx_matrix_bytes(2, 3, 0, ctypes.byref(n), ctypes.byref(n)) == SHAPE


def test_binding_checks():
    x = torch.zeros(4, 64)
    q = nf.quantized_empty(4, 64, "mxfp8", device="cpu")
    for call in (lambda: nf.quantize(x, "mxfp8"), lambda: nf.dequantize(q), lambda: nf.scaled_product(q, q),
                 lambda: nf.fused_norm_quant_fwd(x, x[0], format="mxfp8")):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    with pytest.raises(ValueError, match="unknown format"):
        nf.quantized_empty(4, 64, "fp7", device="cpu")
    with pytest.raises(ValueError, match="contiguous, of"):
        nf._matrix("here", q._replace(codes=q.codes[:3]))
    with pytest.raises(ValueError, match="contiguous, of"):
        nf._matrix("here", q._replace(scales=q.scales.view(torch.uint8)[..., :2]))
    n = nf.quantized_empty(4, 64, "nvfp4", device="cpu")
    with pytest.raises(ValueError, match="mul must be one float32"):
        nf._matrix("here", n._replace(mul=torch.ones(2)))
    with pytest.raises(ValueError, match="mul must be one float32"):
        nf._matrix("here", n._replace(mul=torch.ones(1, dtype=torch.float64)))
    with pytest.raises(ValueError, match="last dimension must be contiguous"):
        nf._plane("here", "x", torch.zeros(4, 6).T)
    with pytest.raises(ValueError, match="matrix"):
        nf._plane("here", "x", torch.zeros(4))
