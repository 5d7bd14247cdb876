"""GPU parity of the group norm (gn_fwd, gn_bwd) against the fp64 oracle.

Bounds, with u = 2^-24 (a rounding of fp32 is off by at most u, relative) and
half the step of the output format on top (2^-8 bf16, 2^-11 fp16, 2^-24 fp32,
relative to the value):

* Sums. A thread adds at most a few hundred values one after the other (n
  additions cost at most n u of the sum of magnitudes; the errors are of both
  signs, so the bound is not met), the merges add a few tens. K = 256 u of the
  sum of magnitudes covers both.
* mean: K u mean|x - k| + u |mean|, k one of the channel's values or a mean of
  some, so for these normal inputs |x - k| <= |x - mean| + 6 std; std <= 1/rstd.
* rstd: half the relative error of var + eps, 2 K u relative. The shift k moves
  with the rows, which bounds it by 164 u for any data of up to 512 rows a
  thread: test_gpu_group_norm_outliers.py derives that and holds rstd to it.
* z: (x - mean) rstd w + beta: the mean's error times rstd |w|, the relative
  error of rstd times |(x - mean) rstd w|, and 4 u of either term.
* activations: |act'| <= 1.13. The exponential is good to (2 + 1.2 |z|) ulp
  of 2 u, quotient and products to 4: (20 + 3 |z|) u of |y|, of which e^-z /
  (1 + e^-z) <= 1 enters. act' in the backward: (30 + 5 |z|) u, absolute.
  The Gaussian distribution function is good to 12 + 1.5 z^2 roundings,
  relative, in its lower tail: (20 + 2 z^2) u of |y| (z^2 and the rest of its
  tail fall below 2^-126 from z = -13 on).
* dx = rstd (w dz - c1 - xhat c2): K u of the sums that c1 and c2 are, 8 u of
  every term, and act' errors times rstd |w dy|.
* dgamma, dbeta: K u of the sum of magnitudes plus act' errors.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

from _blocks import DTYPES, HALF, TINY, U, Padded, f64, make, within
from oracle import group_norm_bwd, group_norm_fwd

pytestmark = pytest.mark.gpu
K = 256 * U


def act_error(z, act):
    """(relative error of act(z), absolute error of act'(z)), arithmetic alone."""
    az = np.minimum(np.abs(z), 200.0)
    if act == "silu":
        return (20 + 3 * az) * U, (30 + 5 * az) * U
    if act == "gelu":
        return (20 + 2 * az * az) * U, (30 + 5 * az) * U
    return 0.0 * az, 0.0 * az


def inputs(rng, dtype, N, R, C, per_sample=False, zero_centered=False, mean=0.0, std=1.5,
           affine=True):
    x = make(rng, (N, R, C), dtype, std, mean + 0.5 * rng.standard_normal((N, 1, C)))
    shape = (N, C) if per_sample else (C,)
    g = make(rng, shape, dtype, 0.2, 0.0 if zero_centered else 1.0) if affine else None
    b = make(rng, shape, dtype, 0.2) if affine else None
    return x, g, b, make(rng, (N, R, C), dtype)


def fwd_bounds(x64, ref, G, dtype, act, eps):
    N, R, C = x64.shape
    sp = lambda t: np.repeat(t, C // G, axis=1)[:, None, :]  # noqa: E731
    m, rs = ref["mean"], ref["rstd"]
    std = 1 / rs
    tol_m = K * 7 * std + 2 * U * np.abs(m)
    tol_r = 2 * K * rs
    term = np.abs(x64 - sp(m)) * sp(rs) * np.abs(ref["w"])
    dz = sp(tol_m * rs) * np.abs(ref["w"]) + 2 * K * term + 4 * U * (term + np.abs(ref["b"]))
    ra, _ = act_error(ref["z"], act)
    y = ref["y"]
    tol_y = 1.13 * dz + ra * np.abs(y) + HALF[dtype] * np.abs(y) + TINY[dtype]
    return tol_y, tol_m, tol_r


def check_fwd(nf, dtype, x, g, b, G, act, eps=1e-5, zero_centered=False, x_extra=0, y_extra=0,
              offset=0, stream=None):
    xd = Padded(x.shape, DTYPES[dtype], x_extra, offset, data=x)
    yd = Padded(x.shape, DTYPES[dtype], y_extra, offset)
    N = x.shape[0]
    md, rd = (Padded((N, G), torch.float32) for _ in range(2))
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    nf.gn_fwd(xd.t, G, dev(g), dev(b), eps, act, zero_centered, yd.t, md.t, rd.t, stream)
    torch.cuda.synchronize()
    ref = group_norm_fwd(f64(x), G, f64(g), f64(b), eps, act, zero_centered)
    ty, tm, tr = fwd_bounds(f64(x), ref, G, dtype, act, eps)
    within(f64(md.t), ref["mean"], tm, "mean")
    within(f64(rd.t), ref["rstd"], tr, "rstd")
    within(f64(yd.t), ref["y"], ty, "y")
    for p, name in ((xd, "x"), (yd, "y"), (md, "mean"), (rd, "rstd")):
        assert p.intact(), f"wrote outside of {name}"
    return yd.t, md.t, rd.t


def check_bwd(nf, dtype, x, g, b, dy, G, act, eps=1e-5, zero_centered=False, extra=(0, 0, 0),
              offset=0, grad="f32"):
    N, R, C = x.shape
    ref = group_norm_fwd(f64(x), G, f64(g), f64(b), eps, act, zero_centered)
    mean, rstd = (torch.from_numpy(ref[k]).float() for k in ("mean", "rstd"))
    dt = DTYPES[dtype]
    xd, dd = Padded(x.shape, dt, extra[0], offset, data=x), Padded(x.shape, dt, extra[1], offset,
                                                                   data=dy)
    od = Padded(x.shape, dt, extra[2], offset)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    gd = None if g is None else Padded(g.shape, DTYPES[grad])
    bd = None if b is None else Padded(b.shape, DTYPES[grad])
    nf.gn_bwd(dd.t, xd.t, G, dev(g), dev(b), act, zero_centered, mean.cuda(), rstd.cuda(), od.t,
              None if gd is None else gd.t, None if bd is None else bd.t)
    torch.cuda.synchronize()
    r = group_norm_bwd(f64(dy), f64(x), G, f64(g), f64(b), f64(mean), f64(rstd), act, zero_centered)
    sp = lambda t: np.repeat(t, C // G, axis=1)[:, None, :]  # noqa: E731
    rs = sp(f64(rstd))
    z = r["xhat"] * r["w"] + (0 if b is None else np.broadcast_to(f64(b), (N, C))[:, None, :])
    # z's own error moves act' by at most |act''| <= 1 times it
    _, aa = act_error(z, act)
    aa = aa + (4 * U * (np.abs(r["xhat"] * r["w"]) + np.abs(z)) if act != "none" else 0.0)
    edz = np.abs(f64(dy)) * aa + 4 * U * np.abs(r["dz"])          # error of dz
    terms = np.abs(r["w"] * r["dz"])
    gm = lambda t: t.reshape(N, R, G, C // G).mean(axis=(1, 3))  # noqa: E731
    ew = np.abs(r["w"]) * edz
    ax = np.abs(r["xhat"])
    e1 = gm(K * terms + ew)
    e2 = gm((K + 4 * U) * terms * ax + ew * ax)
    c1, c2 = np.abs(gm(r["w"] * r["dz"])), np.abs(gm(r["w"] * r["dz"] * r["xhat"]))
    tol = rs * (ew + sp(e1) + ax * sp(e2) + 8 * U * (terms + sp(c1) + ax * sp(c2)))
    within(f64(od.t), r["dx"], tol + HALF[dtype] * np.abs(r["dx"]) + TINY[dtype], "dx")
    eg = ((K + 4 * U) * np.abs(r["dz"]) * ax + edz * ax).sum(axis=1)
    eb = (K * np.abs(r["dz"]) + edz).sum(axis=1)
    for p, key, e, name in ((gd, "dgamma", eg, "dgamma"), (bd, "dbeta", eb, "dbeta")):
        if p is None:
            continue
        want = r[key]
        if p.t.dim() == 1:
            want, e = want.sum(axis=0), (e + K * np.abs(want)).sum(axis=0)
        within(f64(p.t), want, e + HALF[grad] * np.abs(want) + TINY[grad], name)
        assert p.intact(), f"wrote outside of {name}"
    for p, name in ((xd, "x"), (dd, "dy"), (od, "dx")):
        assert p.intact(), f"wrote outside of {name}"
    return od.t


# (dtype, samples, rows, channels, groups, activation)
SHAPES = [
    ("f16", 2, 256, 320, 32, "silu"),     # the UNet widths, groups of 10, 20 and 40
    ("bf16", 1, 64, 640, 32, "silu"),
    ("f16", 3, 33, 1280, 32, "gelu"),
    ("f32", 2, 100, 320, 32, "silu"),
    ("bf16", 2, 1, 64, 8, "none"),        # one row
    ("f32", 1, 1, 1, 1, "silu"),          # one value
    ("bf16", 3, 5, 33, 3, "gelu"),        # rows that no vector fits
    ("f16", 2, 77, 165, 5, "silu"),
    ("f32", 2, 19, 30, 10, "none"),
    ("bf16", 1, 2000, 8, 8, "silu"),      # one vector, a group a channel
    ("bf16", 2, 50, 1024, 1, "silu"),     # one group in all: wider than a tile
    ("f32", 1, 37, 1500, 3, "gelu"),      # groups wider than a tile that end inside one
    ("bf16", 1, 9, 4104, 1, "none"),
    ("f16", 1, 40, 999, 27, "silu"),      # scalar tiles of whole groups
    ("f32", 1, 23, 1001, 7, "silu"),
    ("bf16", 17, 12, 96, 12, "gelu"),
    ("bf16", 1, 4099, 40, 4, "silu"),     # many rows, ragged
    ("f16", 1, 16384, 16, 2, "silu"),
    ("f32", 2, 301, 512, 512, "none"),    # as many groups as a tile has channels
    ("bf16", 2, 333, 250, 5, "silu"),     # rows aligned to 4 and to 8 bytes, last vectors in part
    ("f16", 3, 65, 20, 4, "gelu"),
    ("bf16", 1, 700, 6, 3, "silu"),
    ("f32", 2, 129, 10, 5, "silu"),
    ("f32", 1, 50, 7, 7, "none"),
    ("bf16", 2, 40, 650, 13, "none"),     # tiles of whole groups, the last one narrower
    ("f16", 1, 29, 1026, 2, "silu"),      # groups wider than a tile, rows aligned to 4 bytes
    ("bf16", 1, 21, 1035, 5, "gelu"),     # and to 2
]


@pytest.mark.parametrize("dtype,N,R,C,G,act", SHAPES)
def test_forward(cuda_lib, dtype, N, R, C, G, act):
    x, g, b, _ = inputs(np.random.default_rng(R + C), dtype, N, R, C)
    check_fwd(cuda_lib, dtype, x, g, b, G, act)


@pytest.mark.parametrize("dtype,N,R,C,G,act", SHAPES)
def test_backward(cuda_lib, dtype, N, R, C, G, act):
    x, g, b, dy = inputs(np.random.default_rng(R + C + 1), dtype, N, R, C)
    check_bwd(cuda_lib, dtype, x, g, b, dy, G, act)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("per_sample", [False, True])
@pytest.mark.parametrize("C,G", [(48, 6), (35, 5)])
def test_affine_forms(cuda_lib, dtype, per_sample, C, G):
    """Zero-centered gammas, parameters of each sample, 16-bit gradients."""
    x, g, b, dy = inputs(np.random.default_rng(5), dtype, 3, 41, C, per_sample, True)
    check_fwd(cuda_lib, dtype, x, g, b, G, "silu", zero_centered=True)
    check_bwd(cuda_lib, dtype, x, g, b, dy, G, "silu", zero_centered=True,
              grad="f32" if dtype == "f32" else dtype)


@pytest.mark.parametrize("have", ["neither", "gamma", "beta"])
def test_missing_parameters(cuda_lib, have):
    x, g, b, dy = inputs(np.random.default_rng(6), "bf16", 2, 30, 64)
    g, b = (g if have == "gamma" else None), (b if have == "beta" else None)
    check_fwd(cuda_lib, "bf16", x, g, b, 4, "silu")
    check_bwd(cuda_lib, "bf16", x, g, b, dy, 4, "silu")


@pytest.mark.parametrize("dtype,C,G,x_extra,y_extra,offset", [
    ("bf16", 64, 8, 32, 0, 0),       # a slice of the channels, still in vectors
    ("bf16", 64, 8, 3, 8, 0),        # rows that are not 16-byte aligned
    ("f16", 40, 4, 0, 24, 0),
    ("f32", 24, 3, 4, 4, 1),         # a base that is not
    ("f16", 64, 8, 0, 0, 1),
])
def test_strides_and_alignment(cuda_lib, dtype, C, G, x_extra, y_extra, offset):
    x, g, b, dy = inputs(np.random.default_rng(7), dtype, 2, 91, C)
    check_fwd(cuda_lib, dtype, x, g, b, G, "silu", x_extra=x_extra, y_extra=y_extra, offset=offset)
    check_bwd(cuda_lib, dtype, x, g, b, dy, G, "gelu", extra=(x_extra, y_extra, 16), offset=offset)


def test_a_slice_of_the_same_buffer(cuda_lib):
    """y goes behind x in one buffer of joined channels: no overlap."""
    nf = cuda_lib
    x, g, b, _ = inputs(np.random.default_rng(8), "bf16", 2, 60, 32)
    buf = torch.zeros(2, 60, 64, dtype=torch.bfloat16, device="cuda")
    buf[..., :32] = x.cuda()
    out = nf.fused_group_norm_fwd(buf[..., :32], 4, g.cuda(), b.cuda(), activation="silu",
                                  out=buf[..., 32:])
    want = nf.fused_group_norm_fwd(x.cuda(), 4, g.cuda(), b.cuda(), activation="silu")
    assert torch.equal(buf[..., 32:], want["y"]) and torch.equal(out["mean"], want["mean"])
    assert torch.equal(buf[..., :32], x.cuda())
    with pytest.raises(nf.NormError):
        nf.fused_group_norm_fwd(buf[..., :32], 4, activation="silu", out=buf[..., 31:63])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_mean(cuda_lib, dtype):
    """A mean of 300 standard deviations does not cancel in the variance."""
    rng = np.random.default_rng(9)
    x, g, b, dy = inputs(rng, dtype, 2, 700, 48, mean=450.0)
    check_fwd(cuda_lib, dtype, x, g, b, 6, "none")
    check_bwd(cuda_lib, dtype, x, g, b, dy, 6, "silu")


def test_constant_groups(cuda_lib):
    """No variance: z = beta exactly, in fp32 whatever the constant."""
    x = torch.full((2, 500, 24), 3.7)
    g, b = torch.randn(24), torch.randn(24)
    y, m, r = check_fwd(cuda_lib, "f32", x, g, b, 3, "none")
    assert torch.equal(y.cpu(), b.expand(2, 500, 24))
    assert (m == x[0, 0, 0]).all()


def test_a_group_of_one_value_has_no_gradient(cuda_lib):
    rng = np.random.default_rng(10)
    x, g, b, dy = inputs(rng, "f32", 3, 1, 16)
    assert (check_bwd(cuda_lib, "f32", x, g, b, dy, 16, "silu") == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("C,G", [(64, 8), (33, 3)])
def test_bad_values_stay_in_their_group(cuda_lib, bad, C, G):
    nf = cuda_lib
    x, g, b, dy = inputs(np.random.default_rng(11), "bf16", 2, 90, C)
    run = lambda x, dy: (  # noqa: E731
        nf.fused_group_norm_fwd(x.cuda(), G, g.cuda(), b.cuda(), activation="silu"))
    want = run(x, dy)
    xb = x.clone()
    per = C // G
    xb[1, 40, per + 1] = bad
    got = run(xb, dy)
    assert torch.isnan(got["rstd"][1, 1]) or got["rstd"][1, 1] == 0
    assert torch.isnan(got["y"][1, :, per:2 * per]).all()
    keep = torch.ones(2, 90, C, dtype=torch.bool)
    keep[1, :, per:2 * per] = False
    assert torch.equal(got["y"][keep.cuda()], want["y"][keep.cuda()])
    dyb = dy.clone()
    dyb[1, 40, per + 1] = bad
    grads = [nf.fused_group_norm_bwd(d.cuda(), x.cuda(), G, g.cuda(), b.cuda(), want["mean"],
                                     want["rstd"], activation="silu") for d in (dy, dyb)]
    assert not torch.isfinite(grads[1]["dx"][1, :, per:2 * per]).any()
    assert torch.equal(grads[1]["dx"][keep.cuda()], grads[0]["dx"][keep.cuda()])
    ok = torch.arange(C) != per + 1
    for k in ("dgamma", "dbeta"):
        assert torch.equal(grads[1][k].cpu()[ok], grads[0][k].cpu()[ok])
        assert not torch.isfinite(grads[1][k][per + 1])


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_far_activations(cuda_lib, act, dtype):
    """z out to +-30, where e^-z and the tails are tiny or huge."""
    rng = np.random.default_rng(12)
    x, _, _, dy = inputs(rng, dtype, 1, 200, 32)
    g = torch.full((32,), 10.0).to(DTYPES[dtype])
    b = torch.linspace(-30, 30, 32).to(DTYPES[dtype])
    check_fwd(cuda_lib, dtype, x, g, b, 4, act)
    check_bwd(cuda_lib, dtype, x, g, b, dy, 4, act)


def test_extreme_beta_is_finite(cuda_lib):
    """z = -1000 and 1000: silu and its slope are 0 and z, 0 and 1."""
    nf = cuda_lib
    x = torch.randn(1, 64, 16, device="cuda")
    g, b = torch.ones(16, device="cuda"), torch.full((16,), -1000.0, device="cuda")
    b[8:] = 1000.0
    dy = torch.ones_like(x)
    for act in ("silu", "gelu"):
        f = nf.fused_group_norm_fwd(x, 2, g, b, activation=act)
        assert (f["y"][..., :8] == 0).all() and (f["y"][..., 8:] > 990).all()
        r = nf.fused_group_norm_bwd(dy, x, 2, g, b, f["mean"], f["rstd"], activation=act)
        assert (r["dx"][..., :8] == 0).all() and torch.isfinite(r["dx"]).all()
        assert (r["dbeta"][:8] == 0).all() and (r["dbeta"][8:] == 64).all()


def test_empty(cuda_lib):
    nf = cuda_lib
    g = torch.ones(16, device="cuda")
    for shape in ((0, 5, 16), (3, 0, 16)):
        x = torch.empty(shape, device="cuda")
        f = nf.fused_group_norm_fwd(x, 4, g, g)
        assert f["y"].shape == shape and (f["mean"] == 0).all() and (f["rstd"] == 0).all()
        r = nf.fused_group_norm_bwd(x, x, 4, g, g, f["mean"], f["rstd"])
        assert (r["dgamma"] == 0).all() and (r["dbeta"] == 0).all()


def test_image_layout(cuda_lib):
    """[N, H, W, C], and torch's channels_last through permute."""
    nf = cuda_lib
    x = torch.randn(2, 24, 9, 7, device="cuda").contiguous(memory_format=torch.channels_last)
    g, b = torch.randn(24, device="cuda"), torch.randn(24, device="cuda")
    y = nf.fused_group_norm_fwd(x.permute(0, 2, 3, 1), 4, g, b)["y"]
    want = nf.fused_group_norm_fwd(x.permute(0, 2, 3, 1).reshape(2, 63, 24).contiguous(), 4, g, b)
    assert y.shape == (2, 9, 7, 24) and torch.equal(y.reshape(2, 63, 24), want["y"])
    ref = torch.nn.functional.group_norm(x.double(), 4, g.double(), b.double())
    assert torch.allclose(y.permute(0, 3, 1, 2).double(), ref, atol=1e-5)


def test_same_bits_every_time_and_in_a_graph(cuda_lib):
    """No atomics: the same bits from call to call, on a stream of its own
    and replayed on new inputs; two graphs with workspaces of their own."""
    nf = cuda_lib
    shapes = [(2, 1024, 320, 32), (3, 301, 33, 3)]
    for N, R, C, G in shapes:
        rng = np.random.default_rng(13)
        one, two = (inputs(rng, "bf16", N, R, C) for _ in range(2))
        cuda = [[t.cuda() for t in s] for s in (one, two)]

        def step(x, g, b, dy, wf=None, wb=None):
            f = nf.fused_group_norm_fwd(x, G, g, b, activation="silu", workspace=wf)
            r = nf.fused_group_norm_bwd(dy, x, G, g, b, f["mean"], f["rstd"], activation="silu",
                                        workspace=wb)
            return [f["y"], f["mean"], f["rstd"], r["dx"], r["dgamma"], r["dbeta"]]

        want = [[t.clone() for t in step(*s)] for s in cuda]
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(step(*cuda[0]), want[0]))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        f = nf.fused_group_norm_fwd(cuda[0][0], G, *cuda[0][1:3], activation="silu", stream=side)
        side.synchronize()
        assert torch.equal(f["y"], want[0][0])
        bufs = [[t.clone() for t in cuda[0]] for _ in range(2)]
        graphs = []
        for i in range(2):
            with torch.cuda.stream(side):
                step(*bufs[i])
            torch.cuda.synchronize()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                out = step(*bufs[i])
            graphs.append((gr, out))
        for t, v in zip(bufs[1], cuda[1]):
            t.copy_(v)
        for _ in range(2):
            with torch.cuda.stream(side):
                graphs[1][0].replay()
            graphs[0][0].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(graphs[i][1], want[i]))


def test_workspace_object_is_reused(cuda_lib):
    nf = cuda_lib
    ws = nf.Workspace()
    x = torch.randn(2, 300, 64, device="cuda")
    want = nf.fused_group_norm_fwd(x, 8)["y"]
    assert torch.equal(nf.fused_group_norm_fwd(x, 8, workspace=ws)["y"], want)
    at = ws.buf.data_ptr()
    assert torch.equal(nf.fused_group_norm_fwd(x, 8, workspace=ws)["y"], want)
    assert ws.buf.data_ptr() == at


def test_many_samples_in_batches(cuda_lib):
    """More than one batch of panels: each sample as if it were alone."""
    nf = cuda_lib
    N, R, C, G = 5, 9000, 1024, 32
    x = torch.randn(N, R, C, device="cuda").to(torch.bfloat16)
    x += torch.arange(N, device="cuda").view(N, 1, 1)
    dy = torch.randn(N, R, C, device="cuda").to(torch.bfloat16)
    g, b = (torch.randn(C, device="cuda").to(torch.bfloat16) for _ in range(2))
    f = nf.fused_group_norm_fwd(x, G, g, b, activation="silu")
    r = nf.fused_group_norm_bwd(dy, x, G, g, b, f["mean"], f["rstd"], activation="silu")
    xr = x.double().view(N, R, G, C // G)
    m = xr.mean((1, 3))
    v = (xr - m[:, None, :, None]).square().mean((1, 3))
    assert torch.allclose(f["mean"].double(), m, rtol=1e-5, atol=1e-5)
    assert torch.allclose(f["rstd"].double(), (v + 1e-5).rsqrt(), rtol=1e-5)
    for n in range(N):
        one = slice(n, n + 1)
        xh = ((xr[one] - f["mean"][one, None, :, None].double())
              * f["rstd"][one, None, :, None].double()).view(1, R, C)
        z = xh * g.double() + b.double()
        s = torch.sigmoid(z)
        y = z * s
        assert ((f["y"][one].double() - y).abs() <= 2.0 ** -8 * y.abs() + 1e-5 * (1 + z.abs())).all()
        dz = dy[one].double() * (s + z * s * (1 - s))
        wd = (dz * g.double()).view(1, R, G, -1)
        c1, c2 = wd.mean((1, 3)), (wd * xh.view_as(wd)).mean((1, 3))
        dx = ((wd - c1[:, None, :, None] - xh.view_as(wd) * c2[:, None, :, None])
              * f["rstd"][one, None, :, None].double()).view(1, R, C)
        tol = 2.0 ** -8 * dx.abs() + 1e-4 * (1 + dy[one].double().abs())
        assert ((r["dx"][one].double() - dx).abs() <= tol).all()
