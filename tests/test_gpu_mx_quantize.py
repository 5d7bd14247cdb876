"""The quantiser and its inverse against the oracle, bit for bit."""

import numpy as np
import pytest
import torch

from _blocks import Padded, f64
from _mx import DT, FORMATS, TILED, check_bits, on_gpu
from oracle import mx

pytestmark = pytest.mark.gpu


def data(rng, rows, cols, dtype):
    """Values over many magnitudes, with blocks of zeros, of tiny and of huge
    ones, an infinity and a NaN."""
    v = rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-4, 4, (rows, 1)))
    if rows * cols >= 64:
        flat = v.reshape(-1)
        flat[5:5 + 40] = 0.0
        flat[-30:] *= 1e-30 if dtype != "f16" else 1e-6
        v[rows // 2, :min(cols, 20)] *= 1e4 if dtype == "f16" else 1e30
        v[rows // 3, cols // 2] = np.inf
        v[rows - 1, cols // 3] = np.nan
    return torch.from_numpy(v.astype(np.float32)).to(DT[dtype])


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 17), (130, 100), (128, 256), (257, 1165), (5, 4099)])
def test_codes_and_scales(cuda_lib, fmt, dtype, transpose, rows, cols):
    nf = cuda_lib
    rng = np.random.default_rng(rows * 31 + cols)
    x = data(rng, rows, cols, dtype)
    mul = 0.37 if fmt == "nvfp4" and rows != 3 else None
    for extra, offset in ((0, 0), (3, 1)):
        g = Padded((rows, cols), DT[dtype], extra=extra, offset=offset, data=x.cuda())
        q = nf.quantize(g.t, fmt, mul=on_gpu(mul), transpose=transpose)
        v = f64(x.T if transpose else x)
        check_bits(q, v, fmt, None if mul is None else float(np.float32(mul)))
        assert g.intact()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", FORMATS)
def test_transposes_of_many_tiles(cuda_lib, fmt, dtype):
    """More tiles than the SMs hold at a time, rows of x 16 bytes apart or not."""
    nf = cuda_lib
    rng = np.random.default_rng(8)
    rows, cols = 1101, 5203
    x = data(rng, cols, rows, dtype)
    want = f64(x.T)
    for extra in (11, 0):       # rows of 1112 and of 1101 values
        g = Padded((cols, rows), DT[dtype], extra=extra, data=x.cuda())
        q = nf.quantize(g.t, fmt, transpose=True)
        check_bits(q, want, fmt)
    assert nf.ln_device_error() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_middles_between_codes(cuda_lib, fmt):
    """Quotients that lie on the middle of two codes, for every scale's fraction."""
    nf = cuda_lib
    s = np.arange(8, 16)[:, None, None] / 8.0
    t = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0])
    v = (s * t[None, None, :] * 2.0 ** np.arange(-6.0, 6)[None, :, None]).reshape(96, 16)
    check_bits(nf.quantize(torch.from_numpy(v).float().cuda(), fmt), v, fmt)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", FORMATS)
def test_values(cuda_lib, fmt, dtype):
    nf = cuda_lib
    rng = np.random.default_rng(3)
    for rows, cols in ((1, 1), (5, 50), (131, 300)):
        x = data(rng, rows, cols, "f32")
        mul = 3.3 if fmt == "nvfp4" else None
        q = nf.quantize(x.cuda(), fmt, mul=on_gpu(mul))
        mul = None if mul is None else float(np.float32(mul))
        codes, scales, _ = mx.quantize(f64(x), fmt, mul)
        want = mx.f32(np.where(np.isnan(np.repeat(scales, mx.BLOCK.get(fmt, cols), axis=1)[:, :cols]), np.nan,
                               mx.values(codes, np.where(np.isnan(scales), 1, scales), fmt)))
        want = want if mul is None else mx.f32(want / mul)
        want = torch.from_numpy(want).float().to(DT[dtype])
        g = Padded((rows, cols), DT[dtype], extra=5, offset=1)
        nf.dequantize(q, out=g.t)
        assert torch.equal(torch.nan_to_num(g.t.cpu().float(), nan=-77.0, posinf=1e30, neginf=-1e30),
                           torch.nan_to_num(want.float(), nan=-77.0, posinf=1e30, neginf=-1e30))
        assert g.intact()
        assert torch.equal(torch.nan_to_num(nf.dequantize(q, DT[dtype])), torch.nan_to_num(g.t))


@pytest.mark.parametrize("fmt", FORMATS)
def test_no_byte_outside_is_written_and_padding_is_zero(cuda_lib, fmt):
    """Buffers filled with ones before: every byte of codes and scales is
    written, none around them."""
    nf = cuda_lib
    x = torch.randn(37, 70, device="cuda")
    for transpose in (False, True):
        rows, cols = (70, 37) if transpose else (37, 70)
        nbytes = nf.mx_matrix_bytes(fmt, rows, cols)
        bufs = [torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda") for n in nbytes]
        e = nf.quantized_empty(rows, cols, fmt)
        views = [b[32:32 + n].view(t.dtype).view(t.shape) for b, n, t in zip(bufs, nbytes, (e.codes, e.scales))]
        q = nf.Quantized(*views, fmt, rows, cols)
        nf.mx_quantize(x, q, transpose=transpose)
        check_bits(q, f64(x.T if transpose else x), fmt)
        for b in bufs:
            assert bool((b[:32] == 255).all()) and bool((b[-32:] == 255).all())


def test_expanded_rows_and_one_row(cuda_lib):
    nf = cuda_lib
    x = torch.randn(1, 100, device="cuda")
    for fmt in TILED:
        check_bits(nf.quantize(x.expand(9, 100), fmt), f64(x.expand(9, 100)), fmt)
        assert nf.quantize(x[:0], fmt).codes.numel() == 0


def test_on_another_stream_and_captured(cuda_lib):
    nf = cuda_lib
    x = torch.randn(64, 256, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = nf.quantize(x, "mxfp4", stream=side)
    side.synchronize()
    check_bits(q, f64(x), "mxfp4")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p = nf.quantize(x, "nvfp4", transpose=True)
        y = nf.dequantize(p)
    x.mul_(1.7)
    g.replay()
    check_bits(p, f64(x.T), "nvfp4")
    codes, scales, _ = mx.quantize(f64(x.T), "nvfp4")
    assert np.array_equal(f64(y), mx.values(codes, scales, "nvfp4"))
