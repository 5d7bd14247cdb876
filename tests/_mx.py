"""Helpers of the quantised matrices' tests: matrices from code and scale
values, oracle results as tensors, exact operands."""

from __future__ import annotations

import numpy as np
import torch

from oracle import mx

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FORMATS = mx.FORMATS
TILED = ("mxfp8", "mxfp4", "nvfp4")


def device_matrix(nf, codes, scales, fmt, mul=None):
    """A Quantized on the GPU of code values and scale values (powers of two or
    E4M3 numbers, NaN allowed) of a microscaled format."""
    rows, cols = codes.shape
    odd = np.isnan(scales)
    safe = np.where(odd, 1.0, scales)
    if fmt == "nvfp4":
        stored = np.where(odd, 0x7f, mx.e4m3_bits(safe))
    else:
        stored = np.where(odd, 255, np.log2(safe) + 127)
    q = nf.quantized_empty(rows, cols, fmt, mul=mul)
    q.codes.view(torch.uint8).copy_(torch.from_numpy(mx.pack_codes(codes, fmt)))
    q.scales.view(torch.uint8).copy_(torch.from_numpy(mx.tile(stored.astype(np.uint8))))
    return q


def exact_operand(rng, rows, cols, fmt):
    """(codes, scales) of small whole numbers or halves and scales of 1/2, 1 and
    2: products and sums of thousands of them are fp32 numbers."""
    n = -(-cols // mx.BLOCK[fmt])
    codes = rng.integers(-8, 9, (rows, cols)).astype(float) if fmt == "mxfp8" else \
        rng.choice(np.concatenate((mx.E2M1, -mx.E2M1)), (rows, cols))
    return codes, rng.choice([0.5, 1.0, 2.0], (rows, n))


def random_operand(rng, rows, cols, fmt, std=1.0):
    """(codes, scales, mul) of quantised normal values."""
    v = np.float32(std * rng.standard_normal((rows, cols))).astype(float)
    mul = float(np.float32(2688.0 / np.abs(v).max())) if fmt == "nvfp4" else None
    codes, scales, _ = mx.quantize(v, fmt, mul)
    return codes, scales, mul


def on_gpu(mul):
    return None if mul is None else torch.tensor([mul], dtype=torch.float32, device="cuda")


def check_bits(q, v, fmt, mul=None):
    """Codes and scales of `q` are those of the fp32 values `v`, bit for bit."""
    codes, _, stored = mx.quantize(v, fmt, mul)
    got = q.codes.view(torch.uint8).cpu().numpy()
    want = mx.pack_codes(codes, fmt)
    # the sign of a zero is the value's own and says nothing
    if fmt in ("mxfp4", "nvfp4"):
        def plain(c):
            lo, hi = c & 15, c >> 4
            return np.stack((np.where(lo == 8, 0, lo), np.where(hi == 8, 0, hi)))
    else:
        def plain(c):
            return np.where(c == 128, 0, c)
    assert np.array_equal(plain(got), plain(want)), \
        f"{int((plain(got) != plain(want)).sum())} codes of {want.size}"
    if fmt in TILED:
        assert np.array_equal(q.scales.view(torch.uint8).cpu().numpy(), mx.tile(stored))
    else:
        s = q.scales.cpu().numpy()
        assert np.array_equal(s, stored.reshape(s.shape), equal_nan=True)


def values_of(q):
    """The fp64 values that the bytes of a microscaled Quantized stand for."""
    width = mx.BLOCK[q.format]
    n = -(-q.cols // width)
    codes = q.codes.cpu()
    if q.format == "mxfp8":
        v = codes.double().numpy()
    else:
        c = codes.numpy()
        c = np.stack((c & 15, c >> 4), axis=-1).reshape(q.rows, -1)
        v = np.where(c & 8, -1.0, 1.0) * mx.E2M1[c & 7]
    tiles = q.scales.view(torch.uint8).cpu().numpy()
    s = tiles.transpose(0, 3, 2, 1, 4).reshape(tiles.shape[0] * 128, -1)[:q.rows, :n]
    if q.format == "nvfp4":
        s = torch.from_numpy(np.ascontiguousarray(s)).view(torch.float8_e4m3fn).double().numpy()
    else:
        s = np.where(s == 255, np.nan, 2.0 ** (s.astype(float) - 127))
    return mx.values(v[:, :q.cols], s, q.format, None if q.mul is None else float(q.mul))
