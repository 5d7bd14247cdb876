"""The statistics and y of the norms with quantised results against the oracle, in
every type: the codes are compared with the kernel's own y elsewhere, so y itself,
and the mean that a backward reads, are pinned here."""

import numpy as np
import pytest
import torch

from _blocks import HALF, TINY, U, f64, within
from _mx import DT, FORMATS, on_gpu
from oracle import norm_fwd, round_to_format

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ["layernorm", "rmsnorm"])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,hidden,shift", [(1, 8, 0), (130, 384, 0), (5, 1000, 0), (700, 1160, 0), (2, 8192, 0),
                                               (300, 8192, 0), (3000, 520, 0), (33, 1165, 0), (7, 17, 0), (33, 320, 1),
                                               (3, 8191, 0)])
def test_y_and_statistics(cuda_lib, fmt, dtype, zero, mode, rows, hidden, shift):
    nf = cuda_lib
    rng = np.random.default_rng(hidden + rows)

    def t(*shape, std=1.0, mean=0.0):
        v = torch.from_numpy((mean + std * rng.standard_normal(shape)).astype(np.float32)).to(DT[dtype])
        flat = torch.zeros(v.numel() + shift, dtype=v.dtype, device="cuda")   # off 16 bytes with a shift
        flat[shift:] = v.flatten().cuda()
        return flat[shift:].view(shape)

    x, r, b = t(rows, hidden, mean=0.4), t(rows, hidden), t(hidden, std=0.2)
    gamma, beta = t(hidden, std=0.3, mean=0.0 if zero else 1.0), t(hidden, std=0.5)
    got = nf.fused_norm_quant_fwd(x, gamma, beta, format=fmt, mul=on_gpu(30.0) if fmt == "nvfp4" else None, bias=b,
                                  residual=r, mode=mode, zero_centered_gamma=zero, store_y=True)
    total = round_to_format(round_to_format(f64(x) + f64(b), "f32") + f64(r), "f32")
    s = round_to_format(total, dtype)
    assert np.array_equal(f64(got["sum"]), s)
    rms = mode == "rmsnorm"
    ref = norm_fwd(s, None, None, f64(gamma), None if rms else f64(beta), 1e-5, mode, zero, dtype)
    # A row's sum: at most 64 terms a thread, 10 levels of pairs and 16 warps, 90
    # roundings of the sum of magnitudes; the mean's own division.
    size = np.abs(s).mean(axis=1)
    off = np.zeros(rows) if rms else 92 * U * size
    if rms:
        assert got["mean"] is None
    else:
        within(f64(got["mean"]), ref["mean_exact"], off, "mean")
    within(f64(got["rstd"]), ref["rstd_exact"], 100 * U * ref["rstd_exact"], "rstd")
    # y = (s - mean) rstd w + beta: the mean's error, and the roundings of the
    # difference, of rstd, of 1 + gamma, of the product and of the sum
    w = np.abs(f64(gamma) + (1.0 if zero else 0.0))
    centred = np.abs(s - (0.0 if rms else ref["mean_exact"][:, None])) * ref["rstd_exact"][:, None] * w
    tol = off[:, None] * ref["rstd_exact"][:, None] * w + 105 * U * centred + U * np.abs(ref["y_exact"])
    within(f64(got["y"]), ref["y_exact"], 1.01 * tol + HALF[dtype] * np.abs(ref["y_exact"]) + TINY[dtype], "y")
