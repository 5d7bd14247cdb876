"""Quantised operators where offsets pass 2^31 elements, into buffers that hold
something already, on expanded inputs, and the fast and the general way through
the binding."""

import numpy as np
import pytest
import torch

from _blocks import f64
from _mx import FORMATS, TILED, check_bits, device_matrix, exact_operand, on_gpu
from oracle import mx

pytestmark = pytest.mark.gpu


def raw(q):
    return q.codes.view(torch.uint8), q.scales.view(torch.uint8)


@pytest.mark.parametrize("fmt", ["fp8_row", "mxfp8", "nvfp4"])
def test_rows_past_2_31_elements(cuda_lib, fmt):
    """The last rows of a matrix of 2^31 elements and more are those of the same
    rows alone: norm, quantiser (both ways round) and inverse."""
    nf = cuda_lib
    rows, hidden = (1 << 18) + 133, 8192
    x = torch.empty(rows, hidden, device="cuda", dtype=torch.bfloat16)
    x[:] = torch.randn(hidden, device="cuda").to(torch.bfloat16)
    x[-256:] = torch.randn(256, hidden, device="cuda").to(torch.bfloat16)
    g = torch.ones(hidden, device="cuda", dtype=torch.bfloat16)
    tail = x[-5:].clone()        # rows of a last, partly filled tile of 128
    whole = nf.fused_norm_quant_fwd(x, g, format=fmt, mode="rmsnorm")["q"]
    part = nf.fused_norm_quant_fwd(tail, g, format=fmt, mode="rmsnorm")["q"]
    assert torch.equal(raw(whole)[0][-5:], raw(part)[0])
    assert torch.equal(nf.dequantize(whole, torch.bfloat16)[-5:], nf.dequantize(part, torch.bfloat16))
    del whole
    whole, part = nf.quantize(x, fmt), nf.quantize(tail, fmt)
    assert torch.equal(raw(whole)[0][-5:], raw(part)[0])
    del whole
    # 128 columns of the transpose from the last tile of x's rows
    t = nf.dequantize(nf.quantize(x, fmt, transpose=True), torch.bfloat16)
    if fmt != "fp8_row":         # blocks along the rows: the last ones begin at a multiple of 32
        last = rows // 32 * 32
        want = nf.dequantize(nf.quantize(x[last:], fmt, transpose=True), torch.bfloat16)
        assert torch.equal(t[:, last:], want)


@pytest.mark.parametrize("fmt", TILED)
def test_product_past_2_31_elements(cuda_lib, fmt):
    nf = cuda_lib
    M, N, K = (1 << 18) + 300, 8200, 64
    a = torch.randn(M, K, device="cuda")
    b = nf.quantize(torch.randn(N, K, device="cuda"), fmt)
    r = nf.scaled_product(nf.quantize(a, fmt), b, partials=True)
    part = nf.scaled_product(nf.quantize(a[-4:], fmt), b, partials=True)
    assert torch.equal(r["out"][-4:], part["out"])
    # few rows and many take kernels that add the 128 terms in orders of their own,
    # each within 127 roundings of the sum
    size = torch.nn.functional.pad(part["out"].double().abs(), (0, -N % 128)).view(4, -1, 128).sum(dim=2)
    assert bool(((r["psum"][-4:] - part["psum"]).double().abs() <= 2 * 127 * 2.0 ** -24 * size).all())
    assert nf.ln_device_error() == 0


@pytest.mark.parametrize("hidden", [96, 320, 1001, 2560])
@pytest.mark.parametrize("fmt", FORMATS)
def test_norm_writes_all_of_its_buffers_and_nothing_else(cuda_lib, fmt, hidden):
    nf = cuda_lib
    x, g = torch.randn(37, hidden, device="cuda"), torch.ones(hidden, device="cuda")
    nbytes = nf.mx_matrix_bytes(fmt, 37, hidden)
    bufs = [torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda") for n in nbytes]
    e = nf.quantized_empty(37, hidden, fmt)
    views = [b[32:32 + n].view(t.dtype).view(t.shape) for b, n, t in zip(bufs, nbytes, (e.codes, e.scales))]
    q = nf.Quantized(*views, fmt, 37, hidden)
    y, rstd = torch.empty_like(x), torch.empty(37, device="cuda")
    nf.mx_norm_fwd(x, None, None, g, None, 1e-5, "rmsnorm", False, None, y, None, rstd, q)
    check_bits(q, f64(y), fmt)
    for b in bufs:
        assert bool((b[:32] == 255).all()) and bool((b[-32:] == 255).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_expanded_input_transposed(cuda_lib, fmt):
    nf = cuda_lib
    x = torch.randn(1, 100, device="cuda").expand(300, 100)
    check_bits(nf.quantize(x, fmt, transpose=True), f64(x.T), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_both_ways_through_the_binding(cuda_lib, fmt):
    """A call that allocates in C++ and one that goes through the checks in
    Python (a stream given, outputs given) give the same bytes."""
    nf = cuda_lib
    x, r = (torch.randn(50, 320, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    g = torch.ones(320, device="cuda", dtype=torch.bfloat16)
    b = torch.randn(320, device="cuda", dtype=torch.bfloat16)
    mul = on_gpu(20.0) if fmt == "nvfp4" else None
    here = torch.cuda.current_stream()
    kw = dict(format=fmt, mul=mul, bias=b, residual=r, store_y=True)
    one, two = (nf.fused_norm_quant_fwd(x, g, b, stream=s, **kw) for s in (None, here))
    for k in ("sum", "y", "mean", "rstd"):
        assert torch.equal(one[k], two[k]), k
    assert one["q"][2:5] == two["q"][2:5]
    for t in (False, True):
        p, q = (nf.quantize(x, fmt, mul=mul, transpose=t, stream=s) for s in (None, here))
        assert p.codes.shape == q.codes.shape and p.codes.dtype == q.codes.dtype and p.scales.dtype == q.scales.dtype
        assert all(torch.equal(u, v) for u, v in zip(raw(p), raw(q)))
        assert torch.equal(nf.dequantize(p, torch.float16), nf.dequantize(q, torch.float16, stream=here))
    if fmt in TILED:
        w = nf.quantize(torch.randn(70, 320, device="cuda"), fmt, mul=mul)
        res, bias = torch.randn(50, 70, device="cuda", dtype=torch.float16), torch.randn(70, device="cuda", dtype=torch.float16)
        kw = dict(alpha=0.5, bias=bias, residual=res, dtype=torch.float16, partials=True)
        p, q = (nf.scaled_product(one["q"], w, stream=s, **kw) for s in (None, here))
        for k in ("out", "psum", "psq"):
            assert torch.equal(p[k], q[k]), k
    out = nf.fused_norm_fwd(x, g, b)["y"]
    psum = x.float().sum(dim=1, keepdim=True)
    psq = ((x.float() - psum / 320) ** 2).sum(dim=1, keepdim=True)
    p, q = (nf.fused_norm_fwd_from_partials(x, psum, psq, 320, g, b, kind="sum_m2", stream=s) for s in (None, here))
    assert torch.equal(p["y"], q["y"]) and torch.equal(p["rstd"], q["rstd"]) and out.shape == p["y"].shape


def test_refusals_of_the_binding_on_the_gpu(cuda_lib):
    nf = cuda_lib
    x = torch.randn(8, 64, device="cuda")
    q, p = nf.quantize(x, "mxfp8"), nf.quantize(x, "mxfp4")
    for call, what in (
            (lambda: nf.scaled_product(q, p), nf.NormError),
            (lambda: nf.scaled_product(q, nf.quantize(x[:, :32], "mxfp8")), nf.NormError),
            (lambda: nf.scaled_product(nf.quantize(x, "fp8_row"), nf.quantize(x, "fp8_row")), nf.NormError),
            (lambda: nf.scaled_product(q, q, alpha=float("nan")), nf.NormError),
            (lambda: nf.scaled_product(q, q, bias=torch.zeros(8, device="cuda")), ValueError),      # fp32 with bf16
            (lambda: nf.scaled_product(q, q, residual=torch.zeros(8, 9, device="cuda")), ValueError),
            (lambda: nf.scaled_product(q, q, out=torch.zeros(8, 9, device="cuda")), ValueError),
            (lambda: nf.scaled_product(q, q, dtype=torch.float64), TypeError),
            (lambda: nf.dequantize(q, torch.int32), TypeError),
            (lambda: nf.dequantize(q, out=torch.zeros(7, 64, device="cuda")), ValueError),
            (lambda: nf.quantize(x.double(), "mxfp8"), TypeError),
            (lambda: nf.quantize(x.T, "mxfp8"), ValueError),
            (lambda: nf.quantize(x[None], "mxfp8"), ValueError),
            (lambda: nf.quantize(x, "int8"), ValueError),
            (lambda: nf.quantize(x, "nvfp4", mul=torch.ones(2, device="cuda")), ValueError),
            (lambda: nf.fused_norm_quant_fwd(x, x[0, :32], format="mxfp8"), ValueError),
            (lambda: nf.fused_norm_quant_fwd(x, x[0], format="mxfp8", residual=x[:4]), ValueError),
            (lambda: nf.fused_norm_quant_fwd(x, x[0], format="mxfp8", eps=-1.0), nf.NormError),
            (lambda: nf.fused_norm_quant_fwd(x.T, x[0], format="mxfp8"), ValueError),
            (lambda: nf.fused_norm_quant_fwd(x, x[0].cpu(), format="mxfp8"), ValueError)):
        with pytest.raises(what):
            call()


def test_overflow_and_tiny_values_come_back(cuda_lib):
    """Values past what fp16 holds, and factors that leave fp32's range."""
    nf = cuda_lib
    x = torch.tensor([[3.0e38, 1.0, -2.0e38, 0.0] * 8], device="cuda")
    q = nf.quantize(x, "mxfp8")
    assert bool(nf.dequantize(q, torch.float16)[0, 0].isinf())
    codes, scales, _ = mx.quantize(f64(x), "mxfp8")
    assert np.array_equal(f64(nf.dequantize(q)), mx.values(codes, scales, "mxfp8"))
    n = nf.quantize(torch.full((1, 32), 1e-30, device="cuda"), "nvfp4", mul=on_gpu(1e30))
    assert torch.allclose(nf.dequantize(n), torch.full((1, 32), 1e-30, device="cuda"), rtol=0.07, atol=0)
    big = nf.Quantized(n.codes, n.scales, "nvfp4", 1, 32, on_gpu(1e-39))
    v = nf.dequantize(big)
    assert bool(torch.isinf(v).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hidden", [1, 2, 3, 31, 33, 127, 129, 511, 513, 1025, 4097])
def test_narrow_and_odd_rows(cuda_lib, fmt, hidden):
    nf = cuda_lib
    for rows in (1, 9, 130):
        x = torch.randn(rows, hidden, device="cuda")
        g = 1 + 0.1 * torch.randn(hidden, device="cuda")
        r = nf.fused_norm_quant_fwd(x, g, format=fmt, mode="rmsnorm", store_y=True)
        check_bits(r["q"], f64(r["y"]), fmt)
        for t in (False, True):
            check_bits(nf.quantize(x, fmt, transpose=t), f64(x.T if t else x), fmt)


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(cuda_lib, seed):
    """Sizes over the whole range, each drawn from its logarithm: products of
    whole numbers exactly, codes and scales bit for bit."""
    nf = cuda_lib
    rng = np.random.default_rng(1000 + seed)

    def size(top):
        n = int(np.exp(rng.uniform(0, np.log(top))))
        return max(1, n // (k := int(rng.choice([1, 1, 16, 128]))) * k)

    fmt = TILED[seed % 3]
    M, N, K = size(6000), size(3000), size(1500)
    (ac, as_), (bc, bs) = exact_operand(rng, M, K, fmt), exact_operand(rng, N, K, fmt)
    a, b = device_matrix(nf, ac, as_, fmt), device_matrix(nf, bc, bs, fmt)
    bias = torch.from_numpy(rng.integers(-8, 9, N).astype(np.float32)).cuda()
    res = torch.from_numpy(rng.integers(-8, 9, (M, N)).astype(np.float32)).cuda()
    want, bound = mx.product(mx.values(ac, as_, fmt), mx.values(bc, bs, fmt), 1.0, f64(bias), f64(res))
    assert bound.max() < 2 ** 19      # sums of sixteenths: fp32 numbers
    r = nf.scaled_product(a, b, bias=bias, residual=res, dtype=torch.float32, partials=True)
    assert np.array_equal(f64(r["out"]), want), (M, N, K, fmt)
    for t in range(0, -(-N // 128), 3):
        tile = want[:, 128 * t:128 * t + 128]
        # sums of 128 sixteenths below 2^19 stay fp32 numbers as long as they are below 2^20
        if np.abs(tile).sum(axis=1).max() < 2 ** 20:
            assert np.array_equal(f64(r["psum"][:, t]), tile.sum(axis=1))
    rows, cols, fmt = size(1200), size(3000), FORMATS[seed % 5]
    x = torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).to(
        [torch.float32, torch.bfloat16, torch.float16][seed % 3]).cuda()
    for t in (False, True):
        check_bits(nf.quantize(x, fmt, transpose=t), f64(x.T if t else x), fmt)
    assert nf.ln_device_error() == 0


def test_forks_and_joins_in_a_graph(cuda_lib):
    """Kernels that may be scheduled before what is in front of them has ended:
    behind copies, on a stream that forks from another and joins it again, into
    buffers that the one before still reads, eager and captured."""
    nf = cuda_lib
    rows, hidden, n = 300, 2048, 1536
    src = torch.randn(rows, hidden, device="cuda").to(torch.bfloat16)
    w = torch.randn(n, hidden, device="cuda").to(torch.bfloat16)
    g = torch.ones(hidden, device="cuda", dtype=torch.bfloat16)
    x = torch.empty_like(src)
    side = torch.cuda.Stream()

    def step():
        x.copy_(src)
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            q = nf.quantize(w, "mxfp8")
            q = nf.quantize(nf.dequantize(q, torch.bfloat16), "mxfp8")
        f = nf.fused_norm_quant_fwd(x, g, format="mxfp8", mode="rmsnorm")
        x.zero_()                                # the norm has read it
        here.wait_stream(side)
        out = nf.scaled_product(f["q"], q)["out"]
        keep = out.clone()
        nf.scaled_product(f["q"], q, residual=out, out=out)
        return keep, out, q

    want, twice, _ = (t.clone() if isinstance(t, torch.Tensor) else t for t in step())
    torch.cuda.synchronize()
    q = nf.quantize(nf.dequantize(nf.quantize(w, "mxfp8"), torch.bfloat16), "mxfp8")
    ref = nf.scaled_product(nf.fused_norm_quant_fwd(src, g, format="mxfp8", mode="rmsnorm")["q"], q)["out"]
    torch.cuda.synchronize()
    assert torch.equal(want, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], twice)
    for _ in range(20):
        again = step()
    torch.cuda.synchronize()
    assert torch.equal(again[0], want) and torch.equal(again[1], twice)
