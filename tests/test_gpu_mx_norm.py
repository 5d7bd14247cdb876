"""Norms with quantised results: the stored sum and the statistics against the
oracle, codes and scales bit for bit where y is stored in 32 bits, within half
a step elsewhere."""

import numpy as np
import pytest
import torch

from _blocks import U, f64, within
from _mx import DT, FORMATS, check_bits, on_gpu
from oracle import mx, norm_fwd, round_to_format

pytestmark = pytest.mark.gpu


def run(nf, dtype, rows, hidden, fmt, mode, bias=True, residual=True, zero=False, seed=0, shift=0):
    rng = np.random.default_rng(seed)

    def t(*shape, std=1.0, mean=0.0):
        v = torch.from_numpy((mean + std * rng.standard_normal(shape)).astype(np.float32)).to(DT[dtype])
        if not shift:
            return v.cuda()
        flat = torch.zeros(v.numel() + shift, dtype=v.dtype, device="cuda")   # off 16 bytes
        flat[shift:] = v.flatten().cuda()
        return flat[shift:].view(shape)

    x = t(rows, hidden, mean=0.2)
    b = t(hidden, std=0.1) if bias else None
    r = t(rows, hidden) if residual else None
    gamma = t(hidden, std=0.1, mean=0.0 if zero else 1.0)
    beta = t(hidden, std=0.1) if mode == "layernorm" else None
    mul = on_gpu(30.0) if fmt == "nvfp4" else None
    got = nf.fused_norm_quant_fwd(x, gamma, beta, format=fmt, mul=mul, bias=b, residual=r,
                                  mode=mode, zero_centered_gamma=zero, store_y=True)
    # the sum is formed in fp32: (x + bias) rounded, + residual rounded, then to dtype
    total = f64(x) if b is None else round_to_format(f64(x) + f64(b), "f32")
    total = total if r is None else round_to_format(total + f64(r), "f32")
    ref = norm_fwd(round_to_format(total, dtype), None, None, f64(gamma), f64(beta), 1e-5, mode,
                   zero, dtype)
    return got, ref


def check(nf, got, ref, dtype, fmt, rows, hidden):
    if got["sum"] is not None:
        assert np.array_equal(f64(got["sum"]), ref["sum"])
    # sums of at most 64 terms a thread and 10 levels of pairs: 80 roundings, and
    # those of the division, the root and the mean's part in the squares
    within(f64(got["rstd"]), ref["rstd"], 100 * U * np.abs(ref["rstd"]), "rstd")
    y, q = ref["y_exact"], got["q"]
    mul = 30.0 if fmt == "nvfp4" else None
    if dtype == "f32":
        check_bits(q, f64(got["y"]), fmt, mul)
        return
    codes, scales, _ = mx.quantize(y, fmt, mul)
    step = np.repeat(scales, mx.BLOCK.get(fmt, hidden), axis=1)[:, :hidden] / (mul or 1.0)
    v = f64(nf.dequantize(q))
    slack = 400 * U * (np.abs(y) + np.abs(ref["y_exact"]).max(axis=1, keepdims=True))
    if fmt in ("mxfp4", "nvfp4"):
        tol = np.maximum(0.2 * np.abs(y), 0.25 * step)
    else:
        tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * step)
    # a scale that falls to the other side of a border is a step larger or smaller
    within(v, y, tol * (1 + 2.0 ** -3) + slack, "values")
    exact = mx.values(codes, scales, fmt, mul)
    assert np.mean(np.abs(v - exact) > 1e-5 * np.abs(exact) + slack) < 2e-3 + 2.0 / v.size


@pytest.mark.parametrize("mode", ["layernorm", "rmsnorm"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,hidden", [(1, 8), (3, 320), (130, 384), (5, 1000), (129, 1160), (9, 2560), (2, 8192),
                                         (7, 17), (33, 1165), (3, 8191)])
def test_norm(cuda_lib, fmt, dtype, mode, rows, hidden):
    got, ref = run(cuda_lib, dtype, rows, hidden, fmt, mode, seed=hidden)
    check(cuda_lib, got, ref, dtype, fmt, rows, hidden)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype,hidden", [("bf16", 16384), ("bf16", 16376), ("f16", 40), ("bf16", 128),
                                          ("f32", 4), ("f32", 100), ("bf16", 5120), ("f16", 12288), ("bf16", 1536)])
def test_widths(cuda_lib, fmt, dtype, hidden):
    got, ref = run(cuda_lib, dtype, 131, hidden, fmt, "rmsnorm", bias=False, zero=True)
    check(cuda_lib, got, ref, dtype, fmt, 131, hidden)


@pytest.mark.parametrize("fmt", FORMATS)
def test_operands_left_out_and_unaligned(cuda_lib, fmt):
    for kw in (dict(bias=False), dict(residual=False), dict(bias=False, residual=False), dict(shift=1)):
        got, ref = run(cuda_lib, "bf16", 33, 320, fmt, "layernorm", **kw)
        check(cuda_lib, got, ref, "bf16", fmt, 33, 320)
        assert (got["sum"] is None) == (kw == dict(bias=False, residual=False))


@pytest.mark.parametrize("hidden", [320, 8192, 1165])
def test_rows_that_are_not_finite_or_zero(cuda_lib, hidden):
    """A row's infinity makes its statistics NaN and so all of its scales; a
    row of zeros has zero codes; the others do not change."""
    nf = cuda_lib
    x = torch.randn(6, hidden, device="cuda")
    gamma = torch.ones(hidden, device="cuda")
    bad = x.clone()
    bad[1, 7], bad[2, hidden - 1], bad[4] = float("inf"), float("nan"), 0.0
    for fmt in FORMATS:
        kw = dict(format=fmt, mode="rmsnorm")
        want = nf.dequantize(nf.fused_norm_quant_fwd(x, gamma, **kw)["q"])
        got = nf.dequantize(nf.fused_norm_quant_fwd(bad, gamma, **kw)["q"])
        for r in (0, 3, 5):
            assert torch.equal(got[r], want[r])
        assert bool((got[4] == 0).all())
        assert bool(got[2].isnan().all())
        assert bool(got[1, 7].isnan())


def test_repeats_and_is_captured(cuda_lib):
    nf = cuda_lib
    x, r = (torch.randn(300, 1024, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    gamma = torch.ones(1024, device="cuda", dtype=torch.bfloat16)
    a = nf.fused_norm_quant_fwd(x, gamma, format="mxfp8", residual=r, mode="rmsnorm")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b = nf.fused_norm_quant_fwd(x, gamma, format="mxfp8", residual=r, mode="rmsnorm")
    g.replay()
    torch.cuda.synchronize()
    for k in ("sum", "rstd"):
        assert torch.equal(a[k], b[k])
    assert torch.equal(a["q"].codes.view(torch.uint8), b["q"].codes.view(torch.uint8))
    assert torch.equal(a["q"].scales.view(torch.uint8), b["q"].scales.view(torch.uint8))


def test_no_rows(cuda_lib):
    nf = cuda_lib
    x = torch.empty(0, 64, device="cuda")
    assert nf.fused_norm_quant_fwd(x, torch.ones(64, device="cuda"), format="nvfp4")["q"].codes.numel() == 0
