"""Quantised operators one behind the other on a stream, where each may be
scheduled before the one in front of it has ended: every replay of a captured
run has inputs of its own and is compared with the same calls made one at a
time. A kernel that read too early, or out of a cache that is older than what
was written meanwhile, would see what the replay before left."""

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def source(M, K, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def t(*shape, std=1.0, mean=0.0):
        return (mean + std * torch.randn(shape, generator=gen, device="cuda")).to(BF)

    return {"x": t(M, K, std=1.0 + seed % 3), "g": t(K, std=0.2, mean=1.0), "b": t(K, std=0.5)}


def chain(nf, t, w, fmt, sync):
    """Each call reads what calls just before it wrote: as codes, as x, as the
    residual, as gamma, beta and bias, in place."""
    def go(fn, *a, **k):
        r = fn(*a, **k)
        if sync:
            torch.cuda.synchronize()
        return r

    g = go(nf.dequantize, go(nf.quantize, t["g"][None], fmt), BF)[0]
    b = go(nf.dequantize, go(nf.quantize, t["b"][None], "fp8_row"), BF)[0]
    q = go(nf.quantize, t["x"], fmt)
    o = go(nf.scaled_product, q, w, bias=b, dtype=BF)["out"]
    r = go(nf.dequantize, q, BF)
    f = go(nf.fused_norm_quant_fwd, o, g, b, format=fmt, bias=b, residual=r, store_y=True)
    qt = go(nf.quantize, f["y"], fmt, transpose=True)
    y = go(nf.dequantize, qt, BF)
    q8 = go(nf.quantize, y, "fp8_row")
    q8t = go(nf.quantize, y, "fp8_row", transpose=True)
    q128 = go(nf.quantize, f["sum"], "fp8_block")
    go(nf.scaled_product, f["q"], w, residual=r, out=r)      # the norm has read r
    p = go(nf.scaled_product, f["q"], w, residual=r, dtype=BF, partials=True)
    n = go(nf.fused_norm_quant_fwd, p["out"], g, format="fp8_row", mode="rmsnorm")
    return {"g": g, "b": b, "codes": q.codes, "o": o, "sum": f["sum"], "y": f["y"], "mean": f["mean"],
            "rstd": f["rstd"], "norm codes": f["q"].codes, "norm scales": f["q"].scales,
            "transposed": qt.codes, "transposed scales": qt.scales, "y back": y, "fp8_row": q8.codes,
            "fp8_row scales": q8.scales, "fp8_row transposed": q8t.codes, "fp8_block": q128.codes,
            "in place": r, "out": p["out"], "psum": p["psum"], "psq": p["psq"], "last": n["q"].codes,
            "last scales": n["q"].scales}


def same(got, want, where):
    for k in want:
        a, b = got[k], want[k]
        if a.element_size() == 1:
            a, b = a.view(torch.uint8), b.view(torch.uint8)
        assert torch.equal(a, b), (where, k, int((a != b).sum()))


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,K", [(3000, 2048), (64, 1024), (16, 4096), (777, 1165), (300, 320)])
def test_each_replay_sees_its_own_inputs(cuda_lib, fmt, M, K):
    nf = cuda_lib
    w = nf.quantize(torch.randn(K, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
                    * K ** -0.5, fmt)
    inputs = [source(M, K, s) for s in range(6)]
    want = []
    for i in inputs:
        want.append({k: v.clone() for k, v in chain(nf, i, w, fmt, True).items()})
    static = {k: v.clone() for k, v in inputs[0].items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(nf, static, w, fmt, False)
    for turn in range(3):
        for k, i in enumerate(inputs):
            for n, v in i.items():
                static[n].copy_(v)
            graph.replay()
            torch.cuda.synchronize()
            same(got, want[k], (turn, k))
    # the same behind work that is still under way, so that the calls are all
    # queued before the first one runs
    busy = torch.empty(1 << 29, device="cuda", dtype=torch.float32)
    for k, i in enumerate(inputs):
        for n, v in i.items():
            static[n].copy_(v)
        for _ in range(4):
            busy.fill_(float(k))
        got = chain(nf, static, w, fmt, False)
        torch.cuda.synchronize()
        same(got, want[k], ("eager", k))
    assert nf.ln_device_error() == 0
