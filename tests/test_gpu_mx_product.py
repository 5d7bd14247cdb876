"""The product of microscaled matrices: exact on small whole numbers, within
its roundings on quantised normal values."""

import numpy as np
import pytest
import torch

from _blocks import HALF, Padded, f64, within
from _mx import DT, TILED, device_matrix, exact_operand, on_gpu, random_operand
from oracle import mx

pytestmark = pytest.mark.gpu


def sides(shape_seed, M, N, K, fmt, make):
    rng = np.random.default_rng(shape_seed)
    return make(rng, M, K, fmt), make(rng, N, K, fmt)


SHAPES = [(1, 1, 1), (1, 16, 32), (1, 300, 64), (2, 128, 100), (3, 130, 256), (16, 257, 320), (17, 129, 65),
          (33, 96, 1000), (64, 384, 512), (65, 200, 130), (127, 128, 128), (128, 128, 384), (129, 257, 320),
          (200, 520, 1160), (256, 256, 256), (300, 1165, 96), (513, 300, 2048)]


@pytest.mark.parametrize("fmt", TILED)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_whole_numbers_are_exact(cuda_lib, M, N, K, fmt):
    """Terms are multiples of 1/16 below 256, sums below 2^19: all fp32 numbers."""
    nf = cuda_lib
    (ac, as_), (bc, bs) = sides(M + N + K, M, N, K, fmt, exact_operand)
    a, b = device_matrix(nf, ac, as_, fmt), device_matrix(nf, bc, bs, fmt)
    want, size = mx.product(mx.values(ac, as_, fmt), mx.values(bc, bs, fmt))
    assert size.max() < 2 ** 19
    out = Padded((M, N), torch.float32, extra=3, offset=1)
    nf.scaled_product(a, b, out=out.t)
    got = f64(out.t)
    assert np.array_equal(got, want), f"{int((got != want).sum())} of {want.size}, first {np.argwhere(got != want)[:4].tolist()}"
    assert out.intact()


# More results than single tiles on all SMs hold: pairs of CTAs, both widths.
@pytest.mark.parametrize("fmt", TILED)
@pytest.mark.parametrize("M,N,K", [(2600, 2000, 96), (4100, 4100, 160), (9001, 515, 1000), (3900, 2048, 2100), (140, 20001, 320)])
def test_whole_numbers_are_exact_in_pairs(cuda_lib, M, N, K, fmt):
    test_whole_numbers_are_exact(cuda_lib, M, N, K, fmt)


def bound(want, size, K, dtype):
    """A partial sum is rounded (or cut) once for 16 terms at most often, to 24
    bits, in an order of the hardware's; then the factor, the bias, the residual
    and the rounding to dtype."""
    return HALF[dtype] * np.abs(want) + ((K / 16 + 8) * 2.0 ** -23 + 4 * 2.0 ** -24) * size * (1 + HALF[dtype]) + 2.0 ** -24


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", TILED)
@pytest.mark.parametrize("M,N,K", [(1, 200, 1000), (16, 1024, 4096), (77, 300, 640), (300, 257, 1165), (512, 384, 8192), (2100, 2300, 800), (5000, 4000, 500)])
def test_values(cuda_lib, M, N, K, fmt, dtype):
    nf = cuda_lib
    rng = np.random.default_rng(K)
    (ac, as_, am), (bc, bs, bm) = random_operand(rng, M, K, fmt), random_operand(rng, N, K, fmt, K ** -0.5)
    a, b = device_matrix(nf, ac, as_, fmt, on_gpu(am)), device_matrix(nf, bc, bs, fmt, on_gpu(bm))
    bias = torch.from_numpy(rng.standard_normal(N)).to(DT[dtype]).cuda()
    res = torch.from_numpy(rng.standard_normal((M, N))).to(DT[dtype]).cuda()
    r = nf.scaled_product(a, b, alpha=0.75, bias=bias, residual=res, dtype=DT[dtype], partials=True)
    want, size = mx.product(mx.values(ac, as_, fmt, am), mx.values(bc, bs, fmt, bm), 0.75, f64(bias), f64(res))
    out = f64(r["out"])
    within(out, want, bound(want, size, K, dtype), "out")
    # the statistics are those of what was stored
    for t in range(-(-N // 128)):
        tile = out[:, 128 * t:128 * t + 128]
        n = tile.shape[1]
        s, mean = tile.sum(axis=1), tile.mean(axis=1, keepdims=True)
        # 128 terms in any order, one after the other at worst
        within(f64(r["psum"][:, t]), s, 129 * 2.0 ** -24 * np.abs(tile).sum(axis=1) + 1e-30, "psum")
        m2 = ((tile - mean) ** 2).sum(axis=1)
        off = 130 * 2.0 ** -24 * np.abs(tile).sum(axis=1) / n     # the mean's own error
        within(f64(r["psq"][:, t]), m2, 140 * 2.0 ** -24 * (m2 + (np.abs(tile) * np.abs(tile - mean)).sum(axis=1))
               + 2 * off * np.abs(tile - mean).sum(axis=1) * 2.0 ** -20 + n * off ** 2 + 1e-30, "psq")


@pytest.mark.parametrize("fmt", TILED)
def test_in_place_residual_strides_and_repeats(cuda_lib, fmt):
    nf = cuda_lib
    M, N, K = 150, 200, 320
    (ac, as_), (bc, bs) = sides(1, M, N, K, fmt, exact_operand)
    a, b = device_matrix(nf, ac, as_, fmt), device_matrix(nf, bc, bs, fmt)
    want, _ = mx.product(mx.values(ac, as_, fmt), mx.values(bc, bs, fmt))
    for extra in (0, 5, 8):
        g = Padded((M, N), torch.float32, extra=extra, data=torch.ones(M, N))
        nf.scaled_product(a, b, residual=g.t, out=g.t)
        assert np.array_equal(f64(g.t), want + 1) and g.intact()
    first = nf.scaled_product(a, b)["out"]
    for _ in range(3):
        assert torch.equal(first, nf.scaled_product(a, b)["out"])


@pytest.mark.parametrize("fmt", TILED)
@pytest.mark.parametrize("M", [5, 140])
def test_a_block_that_is_nan_spoils_its_row_alone(cuda_lib, fmt, M):
    nf = cuda_lib
    N, K = 150, 300
    (ac, as_), (bc, bs) = sides(2, M, N, K, fmt, exact_operand)
    clean = nf.scaled_product(device_matrix(nf, ac, as_, fmt), device_matrix(nf, bc, bs, fmt), dtype=torch.float32)["out"]
    as_[3, 1] = np.nan
    bs[7, 0] = np.nan
    out = nf.scaled_product(device_matrix(nf, ac, as_, fmt), device_matrix(nf, bc, bs, fmt), dtype=torch.float32)["out"]
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[3], bad[:, 7] = True, True
    assert torch.equal(out.isnan(), bad)
    assert torch.equal(out[~bad], clean[~bad])


def test_empty(cuda_lib):
    nf = cuda_lib
    for M, N in ((0, 5), (5, 0)):
        a, b = nf.quantized_empty(M, 64, "mxfp4"), nf.quantized_empty(N, 64, "mxfp4")
        assert nf.scaled_product(a, b)["out"].shape == (M, N)
