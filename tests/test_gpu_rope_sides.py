"""Rotary positions whose two sides differ: a norm on one of them alone, one
side given alone. Bounds as in test_gpu_rope.py."""

import numpy as np
import pytest
import torch

from _blocks import DTYPES, HALF, TINY, U, f64, make, within
from oracle import rope_angles, rope_bwd, rope_fwd
from test_gpu_rope import pair_size

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("normed", ["q", "k"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,Hk,D,rot", [(1, 8, 2, 64, 64), (45, 5, 3, 40, 24), (700, 2, 1, 128, 128),
                                          (19, 3, 3, 300, 300)])
def test_a_norm_on_one_side(cuda_lib, dtype, normed, interleaved, T, H, Hk, D, rot):
    """And none on the other, in one call; forward and backward."""
    nf, B, rng = cuda_lib, 2, np.random.default_rng(T + D)
    pos = 1000 + np.arange(T)[None, None].repeat(B, 1)
    freqs = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    th = rope_angles(pos, freqs[None])
    x = {n: make(rng, (B, T, h, D), dtype) for n, h in (("q", H), ("k", Hk))}
    d = {n: make(rng, (B, T, h, D), dtype) for n, h in (("q", H), ("k", Hk))}
    g = make(rng, (D,), dtype, 0.2, 1.0)
    gam = {n: g if n == normed else None for n in ("q", "k")}
    p, f = torch.from_numpy(pos[0]).cuda(), torch.from_numpy(freqs).cuda()
    kw = {f"{normed}_gamma": g.cuda(), "interleaved": interleaved, "eps": 1e-6}
    got = nf.fused_rope_fwd(x["q"].cuda(), x["k"].cuda(), p, f, **kw)
    back = nf.fused_rope_bwd(d["q"].cuda(), d["k"].cuda(), p, f, **{normed: x[normed].cuda()}, **kw)
    torch.cuda.synchronize()
    for n in ("q", "k"):
        okw = dict(gamma=f64(gam[n]), eps=1e-6, interleaved=interleaved)
        r = rope_fwd(f64(x[n]), th, rot, **okw)
        tol = 48 * U * pair_size(r["u"], rot, interleaved, 1.0) + HALF[dtype] * np.abs(r["y"])
        within(f64(got[n]), r["y"], tol + TINY[dtype], n)
        r = rope_bwd(f64(d[n]), f64(x[n]), th, rot, **okw)
        terms = size = pair_size(f64(d[n]), rot, interleaved, 1.0)
        if n == normed:
            x64, w = f64(x[n]), np.abs(f64(g))
            rstd = 1 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + 1e-6)
            xh = np.abs(x64) * rstd
            terms = rstd * (size * w + xh * (size * w * xh).mean(-1, keepdims=True))
            # 1400 rows of heads at most over 300 CTAs' partials: a thread adds few
            tol = 256 * U * (size * xh).sum(axis=(0, 1, 2)) + HALF["f32"] * np.abs(r["dgamma"])
            within(f64(back[f"d{n}_gamma"]), r["dgamma"], tol, f"d{n}_gamma")
        else:
            assert back[f"d{n}_gamma"] is None
        tol = 96 * U * terms + HALF[dtype] * np.abs(r["dx"]) + TINY[dtype]
        within(f64(back["d" + n]), r["dx"], tol, "d" + n)


def test_what_a_side_lacks(cuda_lib):
    """A buffer for the keys without keys is not left unwritten in silence."""
    nf = cuda_lib
    q = torch.randn(2, 5, 3, 16, device="cuda")
    pos, (f, _) = torch.arange(5, device="cuda"), nf.rope_frequencies(16)
    g, out = torch.ones(16, device="cuda"), torch.empty_like(q)
    for call in (lambda: nf.fused_rope_fwd(q, None, pos, f, out_k=out),
                 lambda: nf.rope_fwd(q, q, pos, f, None, None, 0.0, False, False, 1.0, out, None),
                 lambda: nf.rope_bwd(q, None, q, None, pos, f, g, g, 0.0, False, False, 1.0, out,
                                     None, torch.empty_like(g), torch.empty_like(g)),
                 lambda: nf.rope_bwd(q, None, q, None, pos, f, g, None, 0.0, False, False, 1.0, out,
                                     torch.empty_like(q), torch.empty_like(g), None),
                 lambda: nf.rope_bwd(q, q, None, None, pos, f, None, None, 0.0, False, False, 1.0,
                                     out, None, None, None)):
        with pytest.raises(ValueError, match="go together"):
            call()
