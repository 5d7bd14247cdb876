"""Which residuals the product takes beside its output in one buffer. What it
accepts ends at the missing device here; where one is visible that is left out."""

import struct

import pytest
import torch

import normalization_fwd_gb300 as nf
from test_mx_abi import BF16, C, C2, CUDA, INVALID, P1, P2, SC, SC2, Y


@pytest.fixture(scope="module")
def lib():
    nf.build_library()
    return nf.load_library()


def call(lib, out, out_row, res, res_row, M=40, N=50, ps=None, pq=None):
    a, b = (struct.pack("@PPPiqq", c, s, 0, 2, n, 64) for c, s, n in ((C, SC, M), (C2, SC2, N)))
    return lib.mx_product(a, b, 1.0, None, res, res_row, out, out_row, ps, pq, None, BF16)


@pytest.mark.parametrize("kw", [
    dict(out=Y, out_row=100, res=Y + 100, res_row=100),          # columns side by side
    dict(out=Y + 100, out_row=100, res=Y, res_row=100),
    dict(out=Y, out_row=150, res=Y + 200, res_row=150),          # with others between them
    dict(out=Y, out_row=50, res=Y, res_row=50),                  # in place
    dict(out=Y, out_row=200, res=Y, res_row=200),
    dict(out=Y, out_row=50, res=Y, res_row=64, M=1),             # one row: strides say nothing
    dict(out=Y, out_row=50, res=None, res_row=(1 << 63) - 1),    # no residual: its row is not looked at
])
@pytest.mark.skipif(torch.cuda.is_available(), reason="the call would be launched on made-up addresses")
def test_accepted(lib, kw):
    assert call(lib, **kw) == CUDA


@pytest.mark.parametrize("kw", [
    dict(out=Y, out_row=100, res=Y + 98, res_row=100),           # one column in both
    dict(out=Y + 98, out_row=100, res=Y, res_row=100),
    dict(out=Y, out_row=100, res=Y + 104, res_row=100),          # the next row's first columns
    dict(out=Y, out_row=100, res=Y + 100, res_row=104),          # rows that drift into one another
    dict(out=Y, out_row=50, res=Y, res_row=64),
    dict(out=Y, out_row=50, res=Y + 2, res_row=50, M=1),
    dict(out=Y, out_row=50, res=P1 + 8, res_row=50, ps=P1, pq=P2),
])
def test_refused(lib, kw):
    assert call(lib, **kw) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(5, 300, 320), (140, 257, 320), (2600, 2000, 96)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_slices_side_by_side(cuda_lib, M, N, K, dtype):
    """Output and residual as columns of one buffer: the results of apart ones, and
    nothing else is written."""
    gen = torch.Generator(device="cuda").manual_seed(N)

    def t(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    a, b = cuda_lib.quantize(t(M, K), "mxfp8"), cuda_lib.quantize(t(N, K), "mxfp8")
    for gap in (0, 3, 16):
        both = t(M, 2 * N + gap).to(dtype)
        before = both.clone()
        want = cuda_lib.scaled_product(a, b, residual=before[:, :N].contiguous(), dtype=dtype, partials=True)
        got = cuda_lib.scaled_product(a, b, residual=both[:, :N], out=both[:, N + gap:], partials=True)
        assert torch.equal(both[:, N + gap:], want["out"])
        assert torch.equal(both[:, :N + gap], before[:, :N + gap])
        # tiles that start anywhere add their statistics in another order than whole ones
        size = torch.nn.functional.pad(want["out"].double().abs(), (0, -N % 128)).view(M, -1, 128).sum(dim=2)
        assert bool(((got["psum"] - want["psum"]).double().abs() <= 2 * 128 * 2.0 ** -24 * size).all())
    assert cuda_lib.ln_device_error() == 0
