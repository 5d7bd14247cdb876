"""GPU parity of the rotary positions (rope_fwd, rope_bwd) against the fp64
oracle.

Bounds, with u = 2^-24 and half the step of the output format on top:

* the angle: the frequency as a 64-bit fraction of a turn is off by 2^-64
  turns a position, its top 32 bits by 2^-33 turns: 2^-30 radians with the
  fp32 rounding of the fraction at most 2^-24 pi; the Taylor series of the rest
  to the nearest quarter turn are good to 2 ulp. 12 u of the pair's size together.
* u = x rstd w: 512 squares at most, 16 in a thread and the rest by a tree:
  32 u relative, with the root, the quotient and two products.
* the rotation: two products and a sum, 4 u of the pair's size.
  48 u of |u0| + |u1| covers all of it.
* the backward: the same for g', then dx = rstd (g - xhat c): c by the same
  kind of sum, 96 u of the sizes of its terms (a rotated term has the size of
  the pair, so |g'| is taken as |dy0| + |dy1|).
* dgamma: a thread adds the heads and tokens of its share one after the other
  (fewer than 200 here): 256 u of the sum of magnitudes, with the same size
  of a pair.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

from _blocks import DTYPES, HALF, TINY, U, Padded, f64, make, within
from oracle import rope_angles, rope_bwd, rope_fwd

pytestmark = pytest.mark.gpu


def pair_size(a, rot, interleaved, scale):
    """|a0| + |a1| of each element's pair, times the scale; |a| where it passes."""
    a = np.abs(a)
    out = a.copy()
    if interleaved:
        s = a[..., 0:rot:2] + a[..., 1:rot:2]
        out[..., 0:rot:2] = out[..., 1:rot:2] = s * abs(scale)
    else:
        s = a[..., :rot // 2] + a[..., rot // 2:rot]
        out[..., :rot // 2] = out[..., rot // 2:rot] = s * abs(scale)
    return out


def view(shape, dtype, storage, data, offset=0):
    """A [B, T, H, D] CUDA view: "separate", "heads" ([B, H, T, D] in memory) or
    "packed" (room behind the heads); and its padded buffer."""
    B, T, H, D = shape
    if storage == "heads":
        p = Padded((B, H, T, D), DTYPES[dtype], 0, offset)
        t = p.t.transpose(1, 2)
    elif storage == "packed":
        p = Padded((B, T, H * D), DTYPES[dtype], 3 * D, offset)
        t = p.t.unflatten(-1, (H, D))
    else:
        p = Padded(shape, DTYPES[dtype], 0, offset)
        t = p.t
    if data is not None:
        t.copy_(data)
    return t, p


def frequencies(rot, axes, rng):
    f = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    if axes == 1:
        return f[None]
    return f[None] * rng.uniform(0.0, 1.0, (axes, rot // 2))


def case(rng, dtype, B, T, H, Hk, D, rot, axes, start, bits=64):
    pos = start + np.arange(T)[None, None, :] + rng.integers(0, 50, (axes, B, 1))
    freqs = frequencies(rot, axes, rng)
    theta = rope_angles(pos, freqs)
    p = torch.from_numpy(pos).to(torch.int64 if bits == 64 else torch.int32).cuda()
    f = torch.from_numpy(freqs).cuda()
    return (p if axes > 1 else p[0]), (f if axes > 1 else f[0]), theta


def check(nf, dtype, B, T, H, Hk, D, rot, interleaved, norm, storage="separate", axes=1, start=0,
          scale=1.0, zero_centered=False, offset=0, bits=64, seed=0, eps=1e-6, grad="f32",
          backward=True):
    rng = np.random.default_rng(seed + D + T)
    pos, freqs, theta = case(rng, dtype, B, T, H, Hk, D, rot, axes, start, bits)
    kw = dict(eps=eps, zero_centered_gamma=zero_centered, interleaved=interleaved, scale=scale)
    x, dy, ins, outs, gam = {}, {}, {}, {}, {}
    for n, heads in (("q", H), ("k", Hk)):
        x[n], dy[n] = (make(rng, (B, T, heads, D), dtype) for _ in range(2))
        gam[n] = make(rng, (D,), dtype, 0.2, 0.0 if zero_centered else 1.0) if norm else None
        ins[n] = view((B, T, heads, D), dtype, storage, x[n], offset)
        outs[n] = view((B, T, heads, D), dtype, storage, None, offset)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    nf.fused_rope_fwd(ins["q"][0], ins["k"][0], pos, freqs, q_gamma=dev(gam["q"]),
                      k_gamma=dev(gam["k"]), out_q=outs["q"][0], out_k=outs["k"][0], **kw)
    torch.cuda.synchronize()
    okw = dict(eps=eps, interleaved=interleaved, scale=scale, zero_centered=zero_centered)
    for n in ("q", "k"):
        r = rope_fwd(f64(x[n]), theta, rot, gamma=f64(gam[n]), **okw)
        tol = (48 * U * pair_size(r["u"], rot, interleaved, scale) + HALF[dtype] * np.abs(r["y"])
               + TINY[dtype])
        within(f64(outs[n][0]), r["y"], tol, n)
        assert ins[n][1].intact() and outs[n][1].intact(), f"wrote outside of {n}"
    if not backward:
        return
    grads = {n: view((B, T, h, D), dtype, storage, dy[n], offset) for n, h in (("q", H), ("k", Hk))}
    got = nf.fused_rope_bwd(grads["q"][0], grads["k"][0], pos, freqs,
                            q=ins["q"][0] if norm else None, k=ins["k"][0] if norm else None,
                            q_gamma=dev(gam["q"]), k_gamma=dev(gam["k"]),
                            grad_dtype=DTYPES[grad], **kw)
    torch.cuda.synchronize()
    for n in ("q", "k"):
        d64, x64 = f64(dy[n]), f64(x[n])
        r = rope_bwd(d64, x64, theta, rot, gamma=f64(gam[n]), **okw)
        size = pair_size(d64, rot, interleaved, scale)
        if norm:
            rstd = 1 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + eps)
            xh = np.abs(x64) * rstd
            w = np.abs(f64(gam[n]) + (1.0 if zero_centered else 0.0))
            terms = rstd * (size * w + xh * (size * w * xh).mean(-1, keepdims=True))
        else:
            terms = size
        tol = 96 * U * terms + HALF[dtype] * np.abs(r["dx"]) + TINY[dtype]
        within(f64(got["d" + n]), r["dx"], tol, "d" + n)
        assert grads[n][1].intact()
        if norm:
            tol = (256 * U * (size * xh).sum(axis=(0, 1, 2)) + HALF[grad] * np.abs(r["dgamma"])
                   + TINY[grad])
            within(f64(got[f"d{n}_gamma"]), r["dgamma"], tol, f"d{n}_gamma")
        else:
            assert got[f"d{n}_gamma"] is None


# (dim, rot): whole vectors, halves of 8 and 4 bytes, odd halves, part of the head
DIMS = [(128, 128), (64, 64), (40, 40), (80, 32), (96, 24), (256, 256), (2, 2), (6, 4), (30, 22),
        (50, 50), (512, 512), (512, 64), (24, 2), (66, 34), (300, 300)]


@pytest.mark.parametrize("D,rot", DIMS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_head_sizes(cuda_lib, D, rot, interleaved, norm):
    for dtype in ("bf16", "f32"):
        check(cuda_lib, dtype, 2, 5, 3, 2, D, rot, interleaved, norm)


# heads that take 2, 4 and 8 slots a lane: element by element, in pairs and in fours of elements
WIDE = [(140, 140), (160, 150), (256, 70), (134, 134), (258, 258), (500, 402), (510, 30), (460, 460),
        (264, 264)]


@pytest.mark.parametrize("D,rot", WIDE)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_wide_heads(cuda_lib, D, rot, interleaved, dtype):
    check(cuda_lib, dtype, 2, 37, 3, 1, D, rot, interleaved, True)
    check(cuda_lib, dtype, 1, 6, 2, 2, D, rot, interleaved, False, offset=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("storage", ["separate", "heads", "packed"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_storage(cuda_lib, dtype, storage, interleaved):
    check(cuda_lib, dtype, 2, 19, 5, 1, 64, 48, interleaved, True, storage)
    check(cuda_lib, dtype, 3, 1, 8, 8, 32, 32, interleaved, False, storage)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_bases_that_are_not_aligned(cuda_lib, dtype, offset, interleaved):
    check(cuda_lib, dtype, 1, 7, 3, 2, 64, 64, interleaved, True, offset=offset)


@pytest.mark.parametrize("B,T,H,Hk", [(1, 1, 1, 1), (64, 1, 32, 8), (1, 700, 1, 1), (3, 33, 12, 4),
                                      (1, 257, 9, 3), (2, 64, 17, 17)])
@pytest.mark.parametrize("norm", [False, True])
def test_tokens_and_heads(cuda_lib, B, T, H, Hk, norm):
    check(cuda_lib, "bf16", B, T, H, Hk, 32, 32, False, norm)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("bits", [32, 64])
def test_axes(cuda_lib, axes, bits):
    check(cuda_lib, "f16", 2, 30, 4, 2, 40, 40, False, True, axes=axes, bits=bits)
    check(cuda_lib, "f32", 1, 30, 4, 2, 64, 32, True, False, axes=axes, bits=bits)


@pytest.mark.parametrize("start", [1 << 20, (1 << 31) - 60, -1000, 10 ** 12])
def test_far_positions(cuda_lib, start):
    """Angles of millions of turns, in fp32 outputs: nothing is lost. Past
    2^31 the positions have 64 bits."""
    bits = 32 if -2 ** 31 <= start < 2 ** 31 - 100 else 64
    check(cuda_lib, "f32", 2, 9, 2, 1, 64, 64, False, False, start=start, bits=bits)
    check(cuda_lib, "f32", 2, 9, 2, 1, 64, 64, True, True, start=start, bits=64)


@pytest.mark.parametrize("scale,zero_centered,grad", [(1.2, True, "bf16"), (0.0, False, "f16"),
                                                      (-1.0, True, "f32")])
def test_scale_and_zero_centered(cuda_lib, scale, zero_centered, grad):
    check(cuda_lib, "bf16", 1, 40, 4, 2, 64, 32, False, True, scale=scale,
          zero_centered=zero_centered, grad=grad)


def test_frequencies_out_of_the_common_range(cuda_lib):
    """Zero, negative, tiny, and over a turn a position."""
    nf = cuda_lib
    f = np.array([[0.0, -0.5, 1e-300, 5.0, 1000.0, -7e4, 2.0 ** 40, 1e-12]])
    pos = np.array([[[0, 1, -3, 12345, 99999]]])
    th = rope_angles(pos, f)
    x = torch.randn(1, 5, 2, 16)
    got = nf.fused_rope_fwd(x.cuda(), None, torch.from_numpy(pos[0]).cuda(),
                            torch.from_numpy(f[0]).cuda())["q"]
    want = rope_fwd(f64(x), th, 16)
    within(f64(got), want["y"], 64 * U * pair_size(f64(x), 16, False, 1.0), "q")


def test_in_place_and_packed(cuda_lib):
    """q and k of one buffer, rotated in place: v stays, and the results are
    those of the call that allocates."""
    nf = cuda_lib
    B, T, H, Hk, D = 2, 50, 6, 2, 64
    buf = torch.randn(B, T, H + 2 * Hk, D, device="cuda").to(torch.bfloat16)
    keep = buf.clone()
    f, _ = nf.rope_frequencies(48)
    pos = torch.arange(T, device="cuda")
    g = torch.randn(D, device="cuda").to(torch.bfloat16)
    for kw in (dict(), dict(q_gamma=g, k_gamma=g)):
        buf.copy_(keep)
        q, k = buf[:, :, :H], buf[:, :, H:H + Hk]
        want = nf.fused_rope_fwd(q, k, pos, f, **kw)
        out = nf.fused_rope_fwd(q, k, pos, f, out_q=q, out_k=k, **kw)
        assert out["q"] is q
        assert torch.equal(q, want["q"]) and torch.equal(k, want["k"])
        assert torch.equal(buf[:, :, H + Hk:], keep[:, :, H + Hk:])
    # the backward in place over its gradients; without a norm it undoes the forward
    d = {"q": torch.randn(B, T, H, D, device="cuda"), "k": torch.randn(B, T, Hk, D, device="cuda")}
    y = nf.fused_rope_fwd(d["q"], d["k"], pos, f)
    want = nf.fused_rope_bwd(y["q"], y["k"], pos, f)
    nf.rope_bwd(y["q"], y["k"], None, None, pos, f, None, None, 0.0, False, False, 1.0, y["q"],
                y["k"], None, None)
    assert torch.equal(y["q"], want["dq"]) and torch.equal(y["k"], want["dk"])
    assert (y["q"] - d["q"]).abs().max() < 1e-5


def test_a_bad_value_stays_in_its_head(cuda_lib):
    """And with no norm, in its pair; what passes through passes as it is."""
    nf = cuda_lib
    f, _ = nf.rope_frequencies(16)
    pos = torch.arange(9, device="cuda")
    for bad in (float("nan"), float("inf")):
        for interleaved in (False, True):
            x = torch.randn(1, 9, 3, 32, device="cuda")
            want = nf.fused_rope_fwd(x, None, pos, f, interleaved=interleaved)["q"]
            xb = x.clone()
            xb[0, 4, 1, 3] = bad       # rotated
            xb[0, 4, 1, 20] = bad      # passes
            got = nf.fused_rope_fwd(xb, None, pos, f, interleaved=interleaved)["q"]
            pair = [2, 3] if interleaved else [3, 11]
            same = torch.ones_like(x, dtype=torch.bool)
            same[0, 4, 1, pair] = False
            same[0, 4, 1, 20] = False
            assert torch.equal(got[same], want[same])
            assert not torch.isfinite(got[0, 4, 1, pair]).any()
            assert (got[0, 4, 1, 20] == bad) if bad == bad else torch.isnan(got[0, 4, 1, 20])
            g = torch.ones(32, device="cuda")
            got = nf.fused_rope_fwd(xb, None, pos, f, q_gamma=g, interleaved=interleaved)["q"]
            ok = torch.ones(1, 9, 3, dtype=torch.bool)
            ok[0, 4, 1] = False
            clean = nf.fused_rope_fwd(x, None, pos, f, q_gamma=g, interleaved=interleaved)["q"]
            assert torch.equal(got[ok.cuda()], clean[ok.cuda()])


def test_no_tokens_and_no_heads(cuda_lib):
    nf = cuda_lib
    f, _ = nf.rope_frequencies(16)
    g = torch.ones(16, device="cuda")
    for shape, n in (((0, 4, 2, 16), 4), ((2, 0, 2, 16), 0), ((2, 4, 0, 16), 4)):
        q = torch.empty(shape, device="cuda")
        out = nf.fused_rope_fwd(q, q, torch.arange(n, device="cuda"), f, q_gamma=g, k_gamma=g)
        assert out["q"].shape == shape
        r = nf.fused_rope_bwd(q, q, torch.arange(n, device="cuda"), f, q=q, k=q, q_gamma=g,
                              k_gamma=g)
        assert (r["dq_gamma"] == 0).all() and (r["dk_gamma"] == 0).all()
    # keys without heads beside queries with some
    q, k = torch.randn(2, 4, 2, 16, device="cuda"), torch.empty(2, 4, 0, 16, device="cuda")
    r = nf.fused_rope_bwd(q, k, torch.arange(4, device="cuda"), f, q=q, k=k, q_gamma=g, k_gamma=g)
    alone = nf.fused_rope_bwd(q, None, torch.arange(4, device="cuda"), f, q=q, q_gamma=g)
    assert torch.equal(r["dq"], alone["dq"]) and torch.equal(r["dq_gamma"], alone["dq_gamma"])
    assert (r["dk_gamma"] == 0).all()


def test_three_dimensions_and_expanded_inputs(cuda_lib):
    nf = cuda_lib
    f, _ = nf.rope_frequencies(32)
    pos = torch.arange(21, device="cuda", dtype=torch.int32)
    q = torch.randn(21, 4, 32, device="cuda")
    a = nf.fused_rope_fwd(q, None, pos, f)["q"]
    b = nf.fused_rope_fwd(q[None], None, pos, f)["q"][0]
    assert torch.equal(a, b)
    one = torch.randn(1, 21, 1, 32, device="cuda")
    a = nf.fused_rope_fwd(one.expand(3, 21, 4, 32), None, pos, f)["q"]
    b = nf.fused_rope_fwd(one, None, pos, f)["q"]
    assert torch.equal(a, b.expand(3, 21, 4, 32))


def test_same_bits_every_time_and_in_a_graph(cuda_lib):
    nf = cuda_lib
    f, s = nf.rope_frequencies(64, scaling="yarn", factor=4.0, original=256)
    pos = torch.arange(300, device="cuda")
    g = torch.randn(64, device="cuda").to(torch.bfloat16)
    new = lambda h: torch.randn(2, 300, h, 64, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, dq, dk = new(8), new(2), new(8), new(2)
    kw = dict(q_gamma=g, k_gamma=g, scale=s)

    def step():
        a = nf.fused_rope_fwd(q, k, pos, f, **kw)
        b = nf.fused_rope_bwd(dq, dk, pos, f, q=q, k=k, **kw)
        return [a["q"], a["k"], *b.values()]

    want = [t.clone() for t in step()]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = nf.fused_rope_fwd(q, k, pos, f, stream=side, **kw)["q"]
    side.synchronize()
    assert torch.equal(out, want[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    # new positions and inputs, replayed twice
    q2, pos2 = new(8), pos + 77
    keep = q.clone()
    q.copy_(q2)
    pos.copy_(pos2)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))
    q.copy_(keep)
    pos.sub_(77)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
