"""Layouts that the C entry points accept, on real buffers: input and output as
slices of one wider tensor."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", ["x", "y"])
@pytest.mark.parametrize("rows", [40, 3000])
def test_group_norm_of_neighbouring_slices(cuda_lib, first, rows):
    """x and y side by side in rows of 128 channels, either one in front."""
    nf = cuda_lib
    gen = torch.Generator(device="cuda").manual_seed(rows)
    buf = torch.randn(2, rows, 128, device="cuda", generator=gen).to(torch.bfloat16)
    g, b = (torch.randn(64, device="cuda", generator=gen).to(torch.bfloat16) for _ in range(2))
    x, y = (buf[..., :64], buf[..., 64:]) if first == "x" else (buf[..., 64:], buf[..., :64])
    keep = x.clone()
    want = nf.fused_group_norm_fwd(keep, 8, g, b, activation="silu")
    got = nf.fused_group_norm_fwd(x, 8, g, b, activation="silu", out=y)
    assert torch.equal(y, want["y"]) and torch.equal(x, keep)
    assert torch.equal(got["mean"], want["mean"]) and torch.equal(got["rstd"], want["rstd"])
