"""The quantised operators in one run, as a layer's training step and as its
serving: norm into a microscaled format, projection with residual and statistics,
next norm, and the gradients of all of it."""

import numpy as np
import pytest
import torch

from _blocks import HALF, U, f64, within
from _mx import TILED, values_of
from oracle import mx, norm_bwd, norm_fwd
from test_gpu_mx_product import bound

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def factor(fmt, t):
    return (2688.0 / t.abs().amax().float()).reshape(1) if fmt == "nvfp4" else None


def inputs(M, N, K, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def t(*shape, std=1.0, mean=0.0):
        return (mean + std * torch.randn(shape, generator=gen, device="cuda")).to(BF)

    return {"x": t(M, K), "r": t(M, K), "g": t(K, std=0.1, mean=1.0), "w": t(N, K, std=K ** -0.5),
            "skip": t(M, N), "g2": t(N, std=0.1, mean=1.0), "b2": t(N, std=0.1), "dz": t(M, N)}


def forward(nf, i, w, fmt):
    mul = torch.full((1,), 100.0, device="cuda") if fmt == "nvfp4" else None
    f = nf.fused_norm_quant_fwd(i["x"], i["g"], format=fmt, mul=mul, residual=i["r"], mode="rmsnorm")
    p = nf.scaled_product(f["q"], w, residual=i["skip"], dtype=BF, partials=True)
    z = nf.fused_norm_fwd_from_partials(p["out"], p["psum"], p["psq"], p["tile_cols"], i["g2"], i["b2"],
                                        kind="sum_m2")
    return f, p, z


def backward(nf, i, f, p, z, wt, fmt):
    second = nf.fused_norm_bwd(i["dz"], p["out"], i["g2"], z["mean"], z["rstd"])
    do = second["dx"]
    mul = factor(fmt, do)
    dq, dqt = nf.quantize(do, fmt, mul=mul), nf.quantize(do, fmt, mul=mul, transpose=True)
    dy = nf.scaled_product(dq, wt, dtype=BF)["out"]
    y = nf.dequantize(f["q"], BF)
    yt = nf.quantize(y, fmt, mul=f["q"].mul, transpose=True)
    dw = nf.scaled_product(dqt, yt, dtype=torch.float32)["out"]
    first = nf.fused_norm_bwd(dy, f["sum"], i["g"], None, f["rstd"], mode="rmsnorm")
    return {"do": do, "dq": dq, "dqt": dqt, "dy": dy, "yt": yt, "dw": dw, "dx": first["dx"],
            "dgamma": first["dgamma"], "dskip": do}


@pytest.mark.parametrize("fmt", TILED)
@pytest.mark.parametrize("M,N,K", [(1, 256, 320), (40, 320, 1160), (200, 384, 320)])
def test_training_step(cuda_lib, fmt, M, N, K):
    nf = cuda_lib
    i = inputs(M, N, K)
    wmul = factor(fmt, i["w"])
    w, wt = nf.quantize(i["w"], fmt, mul=wmul), nf.quantize(i["w"], fmt, mul=wmul, transpose=True)
    f, p, z = forward(nf, i, w, fmt)
    b = backward(nf, i, f, p, z, wt, fmt)
    # each step on what the one before left
    ref = norm_fwd(f64(i["x"]), None, f64(i["r"]), f64(i["g"]), None, 1e-5, "rmsnorm", False, "bf16")
    assert np.array_equal(f64(f["sum"]), ref["sum"])
    want, size = mx.product(values_of(f["q"]), values_of(w), residual=f64(i["skip"]))
    within(f64(p["out"]), want, bound(want, size, K, "bf16"), "out")
    o = f64(p["out"])
    ref2 = norm_fwd(o, None, None, f64(i["g2"]), f64(i["b2"]), 1e-5, "layernorm", False, "bf16")
    row = np.abs(ref2["y_exact"]).max(axis=1, keepdims=True)
    within(f64(z["y"]), ref2["y_exact"], HALF["bf16"] * np.abs(ref2["y_exact"]) + 400 * U * row, "z")
    for name, left, right, depth in (("dy", b["dq"], wt, N), ("dw", b["dqt"], b["yt"], M)):
        want, size = mx.product(values_of(left), values_of(right))
        within(f64(b[name]), want, bound(want, size, depth, "bf16" if name == "dy" else "f32"), name)
    rb = norm_bwd(f64(b["dy"]), f64(f["sum"]), f64(i["g"]), None, f64(f["rstd"]), "rmsnorm", False, "bf16")
    scale = np.abs(rb["dx_exact"]).max(axis=1, keepdims=True)
    within(f64(b["dx"]), rb["dx_exact"], HALF["bf16"] * np.abs(rb["dx_exact"]) + 400 * U * scale, "dx")
    # and the whole against the gradients without quantisation, within what the
    # operands' own rounding explains: |A B - A' B'| <= |A - A'| |B|_2 + |A'| |B - B'|_2
    # in Frobenius norms and spectral ones
    do, W = f64(b["do"]), f64(i["w"])
    norm2 = lambda a: np.linalg.norm(a, 2)  # noqa: E731
    for name, a, c, qa, qc in (("dy", do, W.T, values_of(b["dq"]), values_of(wt)),
                               ("dw", do.T, f64(nf.dequantize(f["q"])).T, values_of(b["dqt"]), values_of(b["yt"]))):
        exact = a @ c.T
        slack = np.linalg.norm(a - qa) * norm2(c) + np.linalg.norm(qa) * norm2(c - qc)
        assert np.linalg.norm(f64(b[name]) - exact) <= slack + 2 ** -8 * np.linalg.norm(exact), name
        assert slack < np.linalg.norm(a) * norm2(c)      # it says something


def test_formula_against_differences():
    """The chain's gradients as the step above forms them, without quantisation,
    against central differences in 64 bits."""
    rng = np.random.default_rng(1)
    M, N, K = 3, 5, 7
    x, W, skip, dz = (rng.standard_normal(s) for s in ((M, K), (N, K), (M, N), (M, N)))
    g, g2, b2 = 1 + 0.1 * rng.standard_normal(K), 1 + 0.1 * rng.standard_normal(N), rng.standard_normal(N)

    def loss(x, W, skip):
        y = norm_fwd(x, None, None, g, None, 1e-5, "rmsnorm", False, "f64")["y_exact"]
        o = mx.product(y, W, residual=skip)[0]
        return (norm_fwd(o, None, None, g2, b2, 1e-5, "layernorm", False, "f64")["y_exact"] * dz).sum()

    f = norm_fwd(x, None, None, g, None, 1e-5, "rmsnorm", False, "f64")
    o = mx.product(f["y_exact"], W, residual=skip)[0]
    s = norm_fwd(o, None, None, g2, b2, 1e-5, "layernorm", False, "f64")
    do = norm_bwd(dz, o, g2, s["mean"], s["rstd"], "layernorm", False, "f64")["dx_exact"]
    dx = norm_bwd(do @ W, x, g, None, f["rstd"], "rmsnorm", False, "f64")["dx_exact"]
    for grad, make in ((dx, lambda d: (x + d, W, skip)), (do.T @ f["y_exact"], lambda d: (x, W + d, skip)),
                       (do, lambda d: (x, W, skip + d))):
        d = rng.standard_normal(grad.shape) * 1e-5
        diff = (loss(*make(d)) - loss(*make(-d))) / 2
        assert abs(diff - (grad * d).sum()) <= 1e-6 * np.abs(grad * d).sum()


@pytest.mark.parametrize("fmt", TILED)
@pytest.mark.parametrize("M", [1, 40, 300])
def test_captured_and_two_at_a_time(cuda_lib, fmt, M):
    """Replays give what the calls give, two runs on two streams too, and the
    padding of the batch (rows behind the last sequence) stays as it was."""
    nf = cuda_lib
    N, K = 512, 320
    a, b = inputs(M, N, K, 1), inputs(M, N, K, 2)
    w = nf.quantize(a["w"], fmt, mul=factor(fmt, a["w"]))
    want = [forward(nf, i, w, fmt) for i in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for k, i in enumerate((a, b)):
            with torch.cuda.stream(streams[k]):
                got[k] = forward(nf, i, w, fmt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = forward(nf, a, w, fmt)
    graph.replay()
    torch.cuda.synchronize()
    for g, h in ((got[0], want[0]), (got[1], want[1]), (captured, want[0])):
        assert torch.equal(g[0]["q"].codes.view(torch.uint8), h[0]["q"].codes.view(torch.uint8))
        assert torch.equal(g[0]["q"].scales.view(torch.uint8), h[0]["q"].scales.view(torch.uint8))
        assert torch.equal(g[1]["out"], h[1]["out"]) and torch.equal(g[1]["psq"], h[1]["psq"])
        assert torch.equal(g[2]["y"], h[2]["y"])
    padded = torch.full((M + 7, N), 7.0, device="cuda", dtype=BF)
    nf.scaled_product(want[0][0]["q"], w, residual=a["skip"], out=padded[:M])
    assert torch.equal(padded[:M], want[0][1]["out"]) and bool((padded[M:] == 7).all())
    assert nf.ln_device_error() == 0


def test_the_same_matrix_on_both_sides(cuda_lib):
    """A Gram matrix: both operands are one."""
    nf = cuda_lib
    x = torch.randn(300, 640, device="cuda")
    q = nf.quantize(x, "mxfp8")
    want, size = mx.product(values_of(q), values_of(q))
    within(f64(nf.scaled_product(q, q, dtype=torch.float32)["out"]), want, bound(want, size, 640, "f32"), "gram")
