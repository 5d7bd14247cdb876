"""Frequencies that are not finite: no fraction of a turn, so the pair's results
are NaN, as its cosine and sine are; all other pairs are as without."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("axes", [1, 3])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (40, 24), (50, 50)])
def test_a_pair_without_an_angle(cuda_lib, bad, axes, interleaved, norm, D, rot):
    nf = cuda_lib
    gen = torch.Generator(device="cuda").manual_seed(D)
    q, dq = (torch.randn(2, 33, 3, D, device="cuda", generator=gen) for _ in range(2))
    g = torch.randn(D, device="cuda", generator=gen)
    pos = torch.randint(-50, 1000, (axes, 2, 33), device="cuda", generator=gen)
    pos[:, :, 4] = 0           # position 0 too
    f = torch.rand(axes, rot // 2, device="cuda", generator=gen, dtype=torch.float64)
    j = 5
    fb = f.clone()
    fb[axes - 1, j] = bad
    if axes == 1:
        pos, f, fb = pos[0], f[0], fb[0]
    kw = dict(interleaved=interleaved, q_gamma=g if norm else None)
    want, got = (nf.fused_rope_fwd(q, None, pos, t, **kw)["q"] for t in (f, fb))
    pair = [2 * j, 2 * j + 1] if interleaved else [j, j + rot // 2]
    keep = torch.ones(D, dtype=torch.bool, device="cuda")
    keep[pair] = False
    assert torch.isnan(got[..., pair]).all()
    assert torch.equal(got[..., keep], want[..., keep])
    back = nf.fused_rope_bwd(dq, None, pos, fb, q=q if norm else None, **kw)
    if norm:       # the norm's own gradient mixes the elements of a head
        assert torch.isnan(back["dq"]).all()
        assert torch.isnan(back["dq_gamma"][pair]).all()
        assert torch.isfinite(back["dq_gamma"][keep]).all()
    else:
        clean = nf.fused_rope_bwd(dq, None, pos, f, **kw)["dq"]
        assert torch.isnan(back["dq"][..., pair]).all()
        assert torch.equal(back["dq"][..., keep], clean[..., keep])
