"""The operators of a diffusion network's level in one run, as they are used:
group norm + SiLU -> projection -> residual -> LayerNorm -> q, k, v -> heads'
RMSNorm and rotary positions on two axes -> scores -> row softmax -> values,
and the backward of all of it. The normalizations, rotations and the softmax
are the library's; the products between them are torch's.

The reference is torch autograd over the same formulas in 64 bits. Bound: each
library step is exact to some 2^-18 relative (their own tests hold them to
less), the chain has seven of them and five matrix products of up to 192 terms
in fp32 on each way, every one of which moves a result by at most about its
condition times that; results are compared by norm at 2e-4, 50 times below
what a wrong formula for any of them costs here (removing a single term of one
gradient costs more than 1e-2).
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

N, SIDE, C, G, H, D = 2, 6, 96, 8, 4, 24
T = SIDE * SIDE
EPS = 1e-5


def parameters(dtype):
    gen = torch.Generator().manual_seed(5)
    r = lambda *s, std=1.0, mean=0.0: (mean + std * torch.randn(*s, generator=gen, dtype=torch.float64))  # noqa: E731
    p = {"x": r(N, T, C, mean=0.3), "gn_g": r(C, std=0.2, mean=1), "gn_b": r(C, std=0.2),
         "w1": r(C, C, std=C ** -0.5), "ln_g": r(C, std=0.2, mean=1), "ln_b": r(C, std=0.2),
         "wqkv": r(C, 3 * H * D, std=C ** -0.5), "q_g": r(D, std=0.2, mean=1),
         "k_g": r(D, std=0.2, mean=1)}
    up = r(N, T, H, D)
    return {k: v.to("cuda", dtype) for k, v in p.items()}, up.to("cuda", dtype)


def positions():
    t = torch.arange(T, device="cuda")
    return torch.stack([t // SIDE, t % SIDE])


def plain(p, freqs):
    """The chain in torch operations."""
    x = p["x"]
    g = x.view(N, T, G, C // G)
    g = (g - g.mean((1, 3), keepdim=True)) / (g.var((1, 3), correction=0, keepdim=True) + EPS).sqrt()
    z = g.reshape(N, T, C) * p["gn_g"] + p["gn_b"]
    y = (z * torch.sigmoid(z)) @ p["w1"] + x
    n = (y - y.mean(-1, keepdim=True)) / (y.var(-1, correction=0, keepdim=True) + EPS).sqrt()
    n = n * p["ln_g"] + p["ln_b"]
    q, k, v = (n @ p["wqkv"]).view(N, T, 3 * H, D).split(H, dim=2)
    angle = (positions().double()[:, :, None] * freqs[:, None]).sum(0)[None, :, None]
    c, s = angle.cos().to(x.dtype), angle.sin().to(x.dtype)

    def turn(u, gamma):
        u = u / (u.square().mean(-1, keepdim=True) + EPS).sqrt() * gamma
        a, b = u[..., :D // 2], u[..., D // 2:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    q, k = turn(q, p["q_g"]), turn(k, p["k_g"])
    prob = torch.softmax(torch.einsum("bthd,bshd->bhts", q, k) / math.sqrt(D), -1)
    return torch.einsum("bhts,bshd->bthd", prob, v)


def run(nf, p, freqs, up=None):
    """The chain through the library; with `up`, the gradient of its output,
    the gradients of everything in `p`."""
    f1 = nf.fused_group_norm_fwd(p["x"], G, p["gn_g"], p["gn_b"], eps=EPS, activation="silu")
    y = f1["y"] @ p["w1"] + p["x"]
    f2 = nf.fused_norm_fwd(y, p["ln_g"], p["ln_b"], eps=EPS)
    qkv = (f2["y"] @ p["wqkv"]).view(N, T, 3 * H, D)
    q, k, v = qkv[:, :, :H], qkv[:, :, H:2 * H], qkv[:, :, 2 * H:]
    kw = dict(q_gamma=p["q_g"], k_gamma=p["k_g"], eps=EPS)
    r = nf.fused_rope_fwd(q, k, positions(), freqs, **kw)
    scores = torch.einsum("bthd,bshd->bhts", r["q"], r["k"]) / math.sqrt(D)
    prob = nf.softmax_fwd(scores.contiguous())
    out = torch.einsum("bhts,bshd->bthd", prob, v)
    if up is None:
        return out
    grads = {}
    dp = torch.einsum("bthd,bshd->bhts", up, v)
    dv = torch.einsum("bhts,bthd->bshd", prob, up)
    ds = prob * (dp - (dp * prob).sum(-1, keepdim=True)) / math.sqrt(D)
    b = nf.fused_rope_bwd(torch.einsum("bhts,bshd->bthd", ds, r["k"]).contiguous(),
                          torch.einsum("bhts,bthd->bshd", ds, r["q"]).contiguous(), positions(),
                          freqs, q=q, k=k, **kw)
    grads["q_g"], grads["k_g"] = b["dq_gamma"], b["dk_gamma"]
    dqkv = torch.cat((b["dq"], b["dk"], dv), 2).view(N, T, 3 * H * D)
    grads["wqkv"] = torch.einsum("btc,bto->co", f2["y"], dqkv)
    dn = dqkv @ p["wqkv"].T
    l = nf.fused_norm_bwd(dn.contiguous(), y, p["ln_g"], f2["mean"], f2["rstd"])
    grads["ln_g"], grads["ln_b"] = l["dgamma"], l["dbeta"]
    dy = l["dx"]
    grads["w1"] = torch.einsum("btc,bto->co", f1["y"], dy)
    g = nf.fused_group_norm_bwd((dy @ p["w1"].T).contiguous(), p["x"], G, p["gn_g"], p["gn_b"],
                                f1["mean"], f1["rstd"], activation="silu")
    grads["gn_g"], grads["gn_b"] = g["dgamma"], g["dbeta"]
    grads["x"] = g["dx"] + dy
    return out, grads


@pytest.fixture()
def no_tf32():
    keep = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield
    torch.backends.cuda.matmul.allow_tf32 = keep


def frequencies(nf):
    f, scale = nf.rope_frequencies(D // 2, 100.0)
    assert scale == 1.0
    return nf.rope_axes(f, f)


def test_outputs_and_gradients(cuda_lib, no_tf32):
    nf = cuda_lib
    freqs = frequencies(nf)
    p, up = parameters(torch.float32)
    out, grads = run(nf, p, freqs, up)
    p64 = {k: v.double().requires_grad_() for k, v in p.items()}
    want = plain(p64, freqs)
    (want * up.double()).sum().backward()
    assert set(grads) == set(p)
    for name, got, ref in [("out", out, want.detach())] + [(k, grads[k], p64[k].grad) for k in p]:
        rel = float((got.double() - ref).norm() / ref.norm())
        assert rel < 2e-4, (name, rel)


def test_gradients_match_differences(cuda_lib, no_tf32):
    """The loss along a random direction of all parameters, both ways by h: the
    difference is exact to h^2 times a third derivative and to the rounding of
    the loss over h, together some 1e-3 of the slope at h = 1e-2."""
    nf = cuda_lib
    freqs = frequencies(nf)
    p, up = parameters(torch.float32)
    _, grads = run(nf, p, freqs, up)
    gen = torch.Generator(device="cuda").manual_seed(7)
    d = {k: torch.randn(v.shape, device="cuda", generator=gen) * v.std() for k, v in p.items()}
    slope = sum(float((grads[k].double() * d[k].double()).sum()) for k in p)
    h = 1e-2
    loss = lambda s: float((run(nf, {k: v + s * h * d[k] for k, v in p.items()}, freqs).double()  # noqa: E731
                            * up.double()).sum())
    size = sum(float((grads[k].double() * d[k].double()).norm()) for k in p)
    assert abs((loss(1) - loss(-1)) / (2 * h) - slope) < 1e-2 * (abs(slope) + size)
