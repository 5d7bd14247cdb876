"""fp64 oracle of the quantised matrices: codes, scales, their tiles and the
product (test infrastructure).

Values are taken as float64 holding fp32 numbers; the decisions that the
kernels take in fp32 (a factor, a quotient) are rounded to fp32 here as well,
so codes and scales are equal bit for bit.
"""

from __future__ import annotations

import numpy as np

from .norm import round_to_e4m3_satfinite, round_to_format

FORMATS = ("fp8_row", "fp8_block", "mxfp8", "mxfp4", "nvfp4")
BLOCK = {"fp8_block": 128, "mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def f32(v):
    return round_to_format(v, "f32")


def round_to_e2m1(v):
    """Nearest of E2M1's values, ties to the even code, 6 at most in magnitude."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(v), 6.0)
    middles = (E2M1[1:] + E2M1[:-1]) / 2
    code = np.searchsorted(middles, a, side="left")     # a middle goes to the lower code ...
    tie = (code < 7) & (a == middles[np.minimum(code, 6)])
    code = code + (tie & (code % 2 == 1))               # ... unless that one is odd
    return np.copysign(E2M1[code], v)


def e4m3_bits(v):
    """Codes of values that are E4M3 numbers."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    _, e = np.frexp(a)
    e = np.maximum(e - 1, -6)
    m = np.rint(np.ldexp(a, 3 - e)).astype(np.int64)    # 8..15, below 8: subnormal
    code = np.where(m >= 8, ((e + 7) << 3) | (m - 8), m)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def e2m1_bits(v):
    a = np.abs(np.asarray(v, np.float64))
    return (np.searchsorted(E2M1, a) | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def exponent(amax, most):
    """The least e >= -127 with amax <= most * 2^e."""
    out = np.full(np.shape(amax), -127, np.int64)
    amax = np.asarray(amax, np.float64)
    some = amax > 0
    e = np.ceil(np.log2(amax[some] / most)).astype(np.int64)
    e = np.where(most * 2.0 ** (e - 1.0) >= amax[some], e - 1, e)
    e = np.where(most * 2.0 ** e < amax[some], e + 1, e)
    out[some] = np.maximum(e, -127)
    return out


def quantize(v, fmt, mul=None):
    """(code values [rows, cols], scales [rows, blocks] as values, the same as
    stored bytes or fp32). NaN scales and zero codes where a block is not finite."""
    v = np.asarray(v, np.float64)
    rows, cols = v.shape
    width = BLOCK.get(fmt, cols)
    n = -(-cols // width)
    b = np.zeros((rows, n * width))
    b[:, :cols] = v if mul is None or fmt != "nvfp4" else f32(v * float(mul))
    b = b.reshape(rows, n, width)
    odd = ~np.isfinite(b).all(axis=2)
    b = np.where(odd[..., None], 0.0, b)
    amax = np.abs(b).max(axis=2)
    if fmt in ("fp8_row", "fp8_block"):
        a = np.maximum(amax, 2.0 ** -100)
        scale = f32(a / 448.0)
        codes = round_to_e4m3_satfinite(f32(b * f32(448.0 / a)[..., None]))
        stored = np.where(odd, np.nan, scale).astype(np.float32)
    elif fmt == "nvfp4":
        scale = round_to_e4m3_satfinite(f32(amax / 6.0))
        with np.errstate(divide="ignore", invalid="ignore"):
            codes = np.where(scale[..., None] > 0, round_to_e2m1(f32(b / scale[..., None])), 0.0)
        stored = np.where(odd, 0x7f, e4m3_bits(scale)).astype(np.uint8)
    else:
        e = exponent(amax, 448.0 if fmt == "mxfp8" else 6.0)
        scale = 2.0 ** e.astype(np.float64)
        q = b / scale[..., None]
        codes = round_to_e4m3_satfinite(q) if fmt == "mxfp8" else round_to_e2m1(q)
        stored = np.where(odd, 255, e + 127).astype(np.uint8)
    codes = np.where(odd[..., None], 0.0, codes)
    return codes.reshape(rows, -1)[:, :cols], np.where(odd, np.nan, scale), stored


def values(codes, scales, fmt, mul=None):
    """What codes and scales (values, [rows, blocks]) stand for."""
    rows, cols = codes.shape
    s = np.repeat(scales, BLOCK.get(fmt, cols), axis=1)[:, :cols]
    v = codes * s
    return v if mul is None or fmt != "nvfp4" else v / float(mul)


def tile(stored):
    """Scale bytes [rows, blocks] in tiles of 128 rows by 4 blocks."""
    rows, n = stored.shape
    out = np.zeros((-(-rows // 128), -(-n // 4), 32, 4, 4), np.uint8)
    r, b = np.arange(rows)[:, None], np.arange(n)[None, :]
    out[r // 128, b // 4, r % 32, r % 128 // 32, b % 4] = stored
    return out


def pack_codes(codes, fmt):
    """Code bytes of code values [rows, cols], rows padded as the library has them."""
    rows, cols = codes.shape
    if fmt in ("fp8_row", "fp8_block"):
        return e4m3_bits(codes)
    wide = np.zeros((rows, -(-cols // 32) * 32))
    wide[:, :cols] = codes
    if fmt == "mxfp8":
        return e4m3_bits(wide)
    bits = e2m1_bits(wide)
    return bits[:, 0::2] | (bits[:, 1::2] << 4)


def product(a, b, alpha=1.0, bias=None, residual=None):
    """alpha a b^T + bias + residual, and the sum of the magnitudes of its terms."""
    out, size = alpha * (a @ b.T), abs(alpha) * (np.abs(a) @ np.abs(b).T)
    for t in (bias, residual):
        if t is not None:
            out, size = out + t, size + np.abs(t)
    return out, size
