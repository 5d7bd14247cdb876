"""Per-sample parameters of the group norm that are one row expanded over the
samples, and those that are slices of a wider tensor."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def tensors(*shapes):
    gen = torch.Generator(device="cuda").manual_seed(sum(map(sum, shapes)))
    return [torch.randn(s, device="cuda", generator=gen) for s in shapes]


def run(nf, x, dy, g, b):
    f = nf.fused_group_norm_fwd(x, 4, g, b, activation="silu")
    r = nf.fused_group_norm_bwd(dy, x, 4, g, b, f["mean"], f["rstd"], activation="silu")
    return f["y"], r["dx"], r["dgamma"], r["dbeta"]


@pytest.mark.parametrize("N", [1, 3])
@pytest.mark.parametrize("which", ["both", "gamma", "beta", "gamma alone"])
def test_expanded_over_the_samples(cuda_lib, N, which):
    """The forward and the gradients of [N, C] parameters, a row each sample."""
    x, dy, g, b = tensors((N, 70, 24), (N, 70, 24), (N, 24), (N, 24))
    if which != "beta":
        g = g[:1].expand(N, 24)
    if which in ("both", "beta"):
        b = b[:1].expand(N, 24)
    if which == "gamma alone":
        b = None
    # has to agree with the same rows laid out
    whole = [None if p is None else p.clone(memory_format=torch.contiguous_format) for p in (g, b)]
    want = run(cuda_lib, x, dy, *whole)
    got = run(cuda_lib, x, dy, g, b)
    for a, w in zip(got, want):
        assert (a is None) == (w is None)
        if w is not None:
            assert a.shape == w.shape and torch.equal(a, w)
    assert got[2].shape == (N, 24)


def test_one_shared_and_one_per_sample(cuda_lib):
    """Is refused, an expanded one beside a shared one in the backward too."""
    nf = cuda_lib
    x, dy, g, b = tensors((3, 70, 24), (3, 70, 24), (3, 24), (24,))
    f = nf.fused_group_norm_fwd(x, 4)
    for p in (g, g[:1].expand(3, 24)):
        with pytest.raises(ValueError, match="both be shared or both per sample"):
            nf.fused_group_norm_bwd(dy, x, 4, p, b, f["mean"], f["rstd"])
    with pytest.raises(ValueError, match="both be shared or both per sample"):
        nf.fused_group_norm_fwd(x, 4, g, b)


def test_halves_of_one_projection(cuda_lib):
    x, dy, e = tensors((3, 70, 24), (3, 70, 24), (3, 48))
    g, b = e.chunk(2, dim=1)
    want = run(cuda_lib, x, dy, g.contiguous(), b.contiguous())
    for got in (run(cuda_lib, x, dy, g, b), run(cuda_lib, x, dy, g.contiguous(), b)):
        assert all(torch.equal(a, w) for a, w in zip(got, want))


def test_dx_of_many_samples(cuda_lib):
    """More samples than the parameters' gradients can have, without those."""
    nf = cuda_lib
    x, dy, g, b = tensors((70000, 2, 8), (70000, 2, 8), (70000, 8), (70000, 8))
    f = nf.fused_group_norm_fwd(x, 2, g, b, activation="silu")
    dx = torch.empty_like(x)
    nf.gn_bwd(dy, x, 2, g, b, "silu", False, f["mean"], f["rstd"], dx, None, None)
    for n in (slice(0, 3), slice(65534, 65538), slice(69990, 70000)):
        r = nf.fused_group_norm_bwd(dy[n], x[n], 2, g[n], b[n], f["mean"][n], f["rstd"][n],
                                    activation="silu")
        assert torch.equal(dx[n], r["dx"])
