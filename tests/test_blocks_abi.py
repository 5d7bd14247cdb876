"""Group norm and rotary positions without a GPU: declared and exported entry
points, refusals on the host (no call below reaches the GPU), the binding's
own checks, and the frequencies."""

import ctypes
import gc
import math
import os
import re
import struct
import weakref

import numpy as np
import pytest
import torch

import normalization_fwd_gb300 as nf

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, ALIGN, SHAPE, UNSUPPORTED, CUDA, WORKSPACE, INVALID, SCRATCH_LIMIT = range(9)
X, DY, G, B, Y, M, R, DG, DB, WS, POS, F = (0x7f0000000000 + i * 0x10000000 for i in range(12))
BF16 = 1


@pytest.fixture(scope="module")
def lib():
    nf.build_library()
    return nf.load_library()


def test_declared_entry_points_are_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "normfuse.h")).read(),
                  flags=re.S)
    names = sorted(set(re.findall(r"^ln_status ((?:gn|rope)_\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(nf.exported_symbols("gn_") + nf.exported_symbols("rope_"))
    for n in names:
        assert hasattr(lib, n), n
    for name, value in (("GN_ACT_NONE", 0), ("GN_ACT_SILU", 1), ("GN_ACT_GELU", 2),
                        ("ROPE_HALF", 0), ("ROPE_INTERLEAVED", 1)):
        assert re.search(rf"{name} = {value}\b", text) and getattr(nf, name) == value


def gn_fwd(lib, x=X, xs=64 * 40, xr=64, g=G, b=B, ps=0, eps=1e-5, act=1, zc=0, y=Y, ys=64 * 40,
           yr=64, m=M, r=R, N=2, rows=40, C=64, groups=8, dt=BF16, ws=WS, wb=1 << 20):
    return lib.gn_fwd(x, xs, xr, g, b, ps, eps, act, zc, y, ys, yr, m, r, None, N, rows, C, groups,
                      dt, ws, wb)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL),
    (dict(y=None), NULL),
    (dict(dt=3), UNSUPPORTED),
    (dict(act=3), UNSUPPORTED),
    (dict(act=-1), UNSUPPORTED),
    (dict(N=-1), SHAPE),
    (dict(rows=-1), SHAPE),
    (dict(rows=1 << 41), SHAPE),
    (dict(N=1 << 31), SHAPE),
    (dict(C=0), SHAPE),
    (dict(C=65536 + 8), SHAPE),
    (dict(groups=0), SHAPE),
    (dict(groups=7), SHAPE),                       # does not divide 64
    (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID),
    (dict(xr=-64), INVALID),
    (dict(ys=-1), INVALID),
    (dict(ps=63), INVALID),                        # samples' parameters would overlap
    (dict(x=X + 1), ALIGN),
    (dict(b=B + 1), ALIGN),
    (dict(m=M + 2), ALIGN),
    (dict(y=X), INVALID),                          # no working in place
    (dict(y=X + 64), INVALID),
    (dict(yr=63), INVALID),                        # rows of y overlap
    (dict(yr=0), INVALID),
    (dict(ys=64), INVALID),                        # samples of y overlap
    (dict(m=X), INVALID),
    (dict(r=M + 4), INVALID),
    (dict(ws=Y), INVALID),
    (dict(y=G), INVALID),
])
def test_gn_fwd_rejects_on_host(lib, kw, want):
    assert gn_fwd(lib, **kw) == want


def test_gn_fwd_slices_of_one_buffer(lib):
    # x and y side by side in rows of 128: the call gets past the overlap
    # check, to the device query or to the missing workspace
    ok = (CUDA, WORKSPACE)
    assert gn_fwd(lib, xs=128 * 40, xr=128, y=X + 128, ys=128 * 40, yr=128, ws=None) in ok
    assert gn_fwd(lib, xs=128 * 40, xr=128, y=X + 126, ys=128 * 40, yr=128, ws=None) == INVALID
    # y in front of x, and in another period
    assert gn_fwd(lib, x=Y + 128, xs=128 * 40, xr=128, ys=128 * 40, yr=128, ws=None) in ok
    assert gn_fwd(lib, xs=192 * 40, xr=192, y=X + 128, ys=128 * 40, yr=128, ws=None) == INVALID


def gn_bwd(lib, dy=DY, ds=64 * 40, dr=64, x=X, xs=64 * 40, xr=64, g=G, b=B, ps=0, act=1, zc=0, m=M,
           r=R, dx=Y, os_=64 * 40, or_=64, dg=DG, db=DB, N=2, rows=40, C=64, groups=8, dt=BF16,
           gdt=0, ws=WS, wb=1 << 20):
    return lib.gn_bwd(dy, ds, dr, x, xs, xr, g, b, ps, act, zc, m, r, dx, os_, or_, dg, db, None, N,
                      rows, C, groups, dt, gdt, ws, wb)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), NULL),
    (dict(x=None), NULL),
    (dict(m=None), NULL),
    (dict(r=None), NULL),
    (dict(dx=None), NULL),
    (dict(dt=-1), UNSUPPORTED),
    (dict(gdt=3), UNSUPPORTED),
    (dict(act=7), UNSUPPORTED),
    (dict(groups=5), SHAPE),
    (dict(dx=Y + 1), ALIGN),
    (dict(dg=DG + 2), ALIGN),
    (dict(gdt=1, dg=DG + 1), ALIGN),
    (dict(dx=X), INVALID),
    (dict(dx=DY), INVALID),
    (dict(or_=8), INVALID),
    (dict(dg=M), INVALID),
    (dict(db=DG + 64), INVALID),
    (dict(ws=X + 16), INVALID),
    (dict(ps=-8), INVALID),
    (dict(ps=64, N=65536, rows=1, xs=0, ds=0, os_=64), SHAPE),
])
def test_gn_bwd_rejects_on_host(lib, kw, want):
    assert gn_bwd(lib, **kw) == want


def test_gn_workspace_query_on_host(lib):
    out = ctypes.c_size_t(5)
    assert lib.gn_workspace_bytes(2, 40, 64, 8, BF16, 0, None) == NULL
    assert lib.gn_workspace_bytes(2, 40, 64, 9, BF16, 0, ctypes.byref(out)) == SHAPE
    assert lib.gn_workspace_bytes(2, 40, 64, 8, 9, 0, ctypes.byref(out)) == UNSUPPORTED
    assert lib.gn_workspace_bytes(0, 40, 64, 8, BF16, 1, ctypes.byref(out)) == OK
    assert out.value == 0


def heads(x=X, y=Y, g=0, h=4, xs=(40 * 4 * 64, 4 * 64, 64), ys=(40 * 4 * 64, 4 * 64, 64)):
    return struct.pack("@PPPq3q3q", x or 0, y or 0, g, h, *xs, *ys)


def positions(p=POS, bits=64, axes=1, st=(0, 0, 1), f=F, rot=64, layout=0, scale=1.0):
    return struct.pack("@Piq3qPqif", p or 0, bits, axes, *st, f or 0, rot, layout, scale)


def rope(lib, q=None, k=None, pos=None, eps=1e-6, batch=2, tokens=40, dim=64, dt=BF16):
    q = heads() if q is None else q
    pos = positions() if pos is None else pos
    return lib.rope_fwd(q or None, k, pos or None, eps, 0, None, batch, tokens, dim, dt)


@pytest.mark.parametrize("kw,want", [
    (dict(q=b""), NULL),
    (dict(pos=b""), NULL),
    (dict(q=heads(x=None)), NULL),
    (dict(q=heads(y=None)), NULL),
    (dict(k=heads(x=None, y=WS)), NULL),
    (dict(pos=positions(p=None)), NULL),
    (dict(pos=positions(f=None)), NULL),
    (dict(dt=4), UNSUPPORTED),
    (dict(pos=positions(bits=16)), UNSUPPORTED),
    (dict(pos=positions(layout=2)), UNSUPPORTED),
    (dict(pos=positions(axes=0)), SHAPE),
    (dict(pos=positions(axes=5)), SHAPE),
    (dict(pos=positions(rot=63)), SHAPE),
    (dict(pos=positions(rot=0)), SHAPE),
    (dict(pos=positions(rot=66)), SHAPE),
    (dict(dim=63), SHAPE),
    (dict(dim=514), SHAPE),
    (dict(batch=-1), SHAPE),
    (dict(tokens=-1), SHAPE),
    (dict(batch=1 << 30, tokens=1 << 30), SHAPE),
    (dict(q=heads(h=-1)), SHAPE),
    (dict(q=heads(h=65537)), SHAPE),
    (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(pos=positions(scale=float("inf"))), INVALID),
    (dict(pos=positions(st=(0, -1, 1))), INVALID),
    (dict(q=heads(xs=(0, -64, 64))), INVALID),
    (dict(q=heads(x=X + 1)), ALIGN),
    (dict(q=heads(g=G + 1)), ALIGN),
    (dict(pos=positions(p=POS + 4)), ALIGN),
    (dict(pos=positions(f=F + 4)), ALIGN),
    (dict(q=heads(y=X + 128)), INVALID),                      # shifted over itself
    (dict(q=heads(y=X, ys=(40 * 256, 64, 40 * 64))), INVALID),  # in place, other strides
    (dict(q=heads(ys=(40 * 256, 256, 32))), INVALID),         # heads of y overlap
    (dict(q=heads(ys=(0, 256, 64))), INVALID),                # batches of y overlap
    (dict(k=heads(x=WS, y=Y)), INVALID),                      # both outputs in one place
    (dict(k=heads(x=WS, y=X)), INVALID),                      # k's output over q's input
    (dict(q=heads(y=POS)), INVALID),
])
def test_rope_fwd_rejects_on_host(lib, kw, want):
    assert rope(lib, **kw) == want


def test_rope_overlap_of_packed_heads(lib):
    """Queries and keys of one projection in place: not refused by the overlap
    check; without a device the call ends at the device query. (With one it
    would run, so the pointers here are never valid: skip.)"""
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible: the call would be launched on these addresses")
    st = (40 * 8 * 64, 8 * 64, 64)
    q = heads(x=X, y=X, h=6, xs=st, ys=st)
    k = heads(x=X + 6 * 128, y=X + 6 * 128, h=2, xs=st, ys=st)
    assert rope(lib, q=q, k=k) == CUDA
    k = heads(x=X + 5 * 128, y=X + 5 * 128, h=2, xs=st, ys=st)
    assert rope(lib, q=q, k=k) == INVALID
    # heads before tokens in memory: [batch, heads, tokens, dim]
    st = (8 * 40 * 64, 64, 40 * 64)
    q = heads(x=X, y=X, h=6, xs=st, ys=st)
    k = heads(x=X + 6 * 40 * 128, y=X + 6 * 40 * 128, h=2, xs=st, ys=st)
    assert rope(lib, q=q, k=k) == CUDA


def heads_grad(dy=DY, x=X, dx=Y, g=G, dg=DG, h=4, ds=None, xs=None, os_=None):
    st = (40 * 4 * 64, 4 * 64, 64)
    return struct.pack("@PPPPPq3q3q3q", dy or 0, x or 0, dx or 0, g or 0, dg or 0, h, *(ds or st),
                       *(xs or st), *(os_ or st))


def rope_b(lib, q=None, k=None, pos=None, gdt=0, ws=WS, wb=1 << 24, tokens=40, dt=BF16):
    q = heads_grad() if q is None else q
    return lib.rope_bwd(q or None, k, pos or positions(), 1e-6, 0, None, 2, tokens, 64, dt, gdt, ws,
                        wb)


@pytest.mark.parametrize("kw,want", [
    (dict(q=b""), NULL),
    (dict(q=heads_grad(dy=None)), NULL),
    (dict(q=heads_grad(dx=None)), NULL),
    (dict(q=heads_grad(x=None)), NULL),                # the norm needs x
    (dict(q=heads_grad(g=None)), INVALID),             # a gradient of no gamma
    (dict(gdt=5), UNSUPPORTED),
    (dict(q=heads_grad(dg=DG + 2)), ALIGN),
    (dict(q=heads_grad(dx=X)), INVALID),               # x is not to be written over
    (dict(q=heads_grad(dx=DY + 256)), INVALID),
    (dict(q=heads_grad(dg=DY)), INVALID),
    (dict(ws=DY), INVALID),
    (dict(ws=None), WORKSPACE),
    (dict(ws=WS + 8), WORKSPACE),
    (dict(k=heads_grad(dy=WS, x=POS, dx=DB, dg=DG)), INVALID),   # one dgamma for both
])
def test_rope_bwd_rejects_on_host(lib, kw, want):
    assert rope_b(lib, **kw) == want


def test_rope_workspace_query_on_host(lib):
    out = ctypes.c_size_t(5)
    assert lib.rope_bwd_workspace_bytes(64, None) == NULL
    assert lib.rope_bwd_workspace_bytes(63, ctypes.byref(out)) == SHAPE
    assert lib.rope_bwd_workspace_bytes(514, ctypes.byref(out)) == SHAPE


def freqs(rot, **kw):
    f, s = nf.rope_frequencies(rot, device="cpu", **kw)
    return f.numpy(), s


def test_frequencies():
    plain, s = freqs(64)
    assert s == 1.0 and plain.dtype == np.float64
    assert np.allclose(plain, 10000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    got, s = freqs(64, scaling="linear", factor=4.0)
    assert s == 1.0 and np.allclose(got, plain / 4, rtol=1e-15)
    got, s = freqs(64, scaling="ntk", factor=4.0)
    assert s == 1.0 and got[0] == 1.0 and math.isclose(got[-1], plain[-1] / 4, rel_tol=1e-12)
    assert freqs(2, scaling="ntk", factor=4.0)[0].tolist() == [1.0]
    got, s = freqs(128, scaling="yarn", factor=8.0, original=16384)
    plain, _ = freqs(128)
    assert math.isclose(s, 0.1 * math.log(8) + 1, rel_tol=1e-6)
    turns = 16384 * plain / (2 * math.pi)
    # what turns clearly over 32 times stays, what turns clearly under once is stretched
    assert np.allclose(got[turns > 40], plain[turns > 40], rtol=1e-14)
    assert np.allclose(got[turns < 0.8], plain[turns < 0.8] / 8, rtol=1e-14)
    between = (turns < 25) & (turns > 1.2)
    assert ((got[between] < plain[between]) & (got[between] > plain[between] / 8)).all()
    assert (np.diff(got) < 0).all()
    assert np.allclose(freqs(64, scaling="yarn", factor=1.0)[0], freqs(64)[0], rtol=1e-14)


@pytest.mark.parametrize("args,kw,status", [
    ((63,), {}, SHAPE), ((0,), {}, None), ((-2,), {}, None), ((514,), {}, SHAPE),
    ((64, 1.0), {}, INVALID), ((64, float("inf")), {}, INVALID), ((64, float("nan")), {}, INVALID),
    ((64,), dict(scaling="linear", factor=0.5), INVALID),
    ((64,), dict(scaling="ntk", factor=float("nan")), INVALID),
    ((64,), dict(scaling="yarn", factor=2.0, original=0), INVALID),
    ((64,), dict(scaling="yarn", factor=2.0, turns_fast=1.0, turns_slow=2.0), INVALID),
    ((64,), dict(scaling="yarn", factor=2.0, turns_slow=0.0), INVALID),
])
def test_frequencies_refuse(args, kw, status):
    with pytest.raises(nf.NormError) as e:
        nf.rope_frequencies(*args, device="cpu", **kw)
    if status is not None:
        assert e.value.status == status
    with pytest.raises(ValueError):
        nf.rope_frequencies(64, scaling="cubic", device="cpu")


def test_axes_table():
    a, b = torch.tensor([1.0, 0.5], dtype=torch.float64), torch.tensor([0.25], dtype=torch.float64)
    assert nf.rope_axes(a, b).tolist() == [[1.0, 0.5, 0.0], [0.0, 0.0, 0.25]]


def test_binding_refuses_host_tensors():
    x, f = torch.zeros(2, 3, 8), torch.ones(4, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        nf.fused_group_norm_fwd(x, 2)
    with pytest.raises(ValueError, match="CUDA"):
        nf.fused_rope_fwd(x, None, torch.arange(2), f)
    with pytest.raises(TypeError):
        nf.fused_rope_bwd([1], None, torch.arange(2), f)


def test_rows_of_strided_tensors():
    rows = nf._rows_of
    x = torch.empty(2, 5, 7, 12)
    assert rows(x, "x") == (2, 35, 12, 420, 12)
    assert rows(x[..., :8], "x") == (2, 35, 8, 420, 12)
    assert rows(x[:, :, 3:4], "x") == (2, 5, 12, 420, 84)
    assert rows(x[:, 2:3], "x") == (2, 7, 12, 420, 12)
    assert rows(torch.empty(3, 8), "x") == (3, 1, 8, 8, 0)
    assert rows(torch.empty(3, 0, 8), "x")[:3] == (3, 0, 8)
    assert rows(torch.empty(2, 12, 5, 7).to(memory_format=torch.channels_last).permute(0, 2, 3, 1),
                "x") == (2, 35, 12, 420, 12)
    for bad in (x[:, :, :5], x.transpose(1, 2), x.permute(0, 3, 1, 2), torch.empty(8)):
        with pytest.raises(ValueError):
            rows(bad, "x")


def test_an_outgrown_workspace_buffer_stays():
    """A graph captured with the smaller buffer still writes to it."""
    w = nf.Workspace("cpu")
    small = weakref.ref(w.take(64))
    at = w.take(32).data_ptr()
    assert w.take(4096).numel() == 4096 and w.take(64).numel() == 4096
    gc.collect()
    assert small() is not None and small().data_ptr() == at != w.take(64).data_ptr()
