"""Group norm and rotary positions where offsets pass 2^31 elements, where a
cluster takes many panels of rows that are aligned to less than 16 bytes, and
with calls at the same time on two streams.

A strided call gets the launch of a compact one of the same shape and
alignment, so the results of the two are compared bit for bit; the compact
ones are held to the fp64 oracle in the operators' own tests. Each large test
holds about 20 GB of device memory and frees it when done.
"""

from __future__ import annotations

import gc

import numpy as np
import pytest
import torch

from test_gpu_group_norm import check_bwd, check_fwd, inputs

pytestmark = pytest.mark.gpu

TWO31 = 2 ** 31


@pytest.fixture(autouse=True)
def _free_device_memory():
    yield
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def spread(shape, strides, data=None, dtype=torch.bfloat16):
    """A view of `shape` whose steps are far apart, in a buffer of its own."""
    need = sum((n - 1) * s for n, s in zip(shape, strides)) + 1
    t = torch.empty(need, dtype=dtype, device="cuda").as_strided(shape, strides)
    if data is not None:
        t.copy_(data)
    return t


@pytest.mark.parametrize("R,strides", [
    (40, (TWO31 + 64, 2 ** 16, 1)),          # samples far apart
    (5, (64, TWO31 // 4 + 128, 1)),          # rows far apart, samples between them
])
def test_group_norm_far_strides(cuda_lib, R, strides):
    nf = cuda_lib
    gen = torch.Generator(device="cuda").manual_seed(3)
    new = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()  # noqa: E731
    x, dy, g, b = new(2, R, 64), new(2, R, 64), new(64), new(64)
    want = nf.fused_group_norm_fwd(x, 8, g, b, activation="silu")
    back = nf.fused_group_norm_bwd(dy, x, 8, g, b, want["mean"], want["rstd"], activation="silu")
    xf, yf = spread(x.shape, strides, x), spread(x.shape, strides)
    got = nf.fused_group_norm_fwd(xf, 8, g, b, activation="silu", out=yf)
    assert torch.equal(yf, want["y"]) and torch.equal(got["mean"], want["mean"])
    assert torch.equal(got["rstd"], want["rstd"])
    df, dg, db = spread(x.shape, strides, dy), torch.empty(64, device="cuda"), torch.empty(
        64, device="cuda")
    nf.gn_bwd(df, xf, 8, g, b, "silu", False, got["mean"], got["rstd"], yf, dg, db)
    assert torch.equal(yf, back["dx"])
    assert torch.equal(dg, back["dgamma"]) and torch.equal(db, back["dbeta"])


@pytest.mark.parametrize("strides", [
    (TWO31 + 512, 512, 64, 1),               # sequences far apart
    (512, TWO31 // 2 + 1024, 64, 1),         # tokens
    (1024, 64, TWO31 // 3 // 8 * 8, 1),      # heads
])
@pytest.mark.parametrize("norm", [False, True])
def test_rope_far_strides(cuda_lib, strides, norm):
    nf = cuda_lib
    gen = torch.Generator(device="cuda").manual_seed(4)
    new = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()  # noqa: E731
    q, dq = new(2, 5, 8, 64), new(2, 5, 8, 64)
    gamma = new(64) if norm else None
    f, scale = nf.rope_frequencies(64)
    pos = torch.arange(1000, 1005, device="cuda")
    want = nf.fused_rope_fwd(q, None, pos, f, q_gamma=gamma, scale=scale)["q"]
    back = nf.fused_rope_bwd(dq, None, pos, f, q=q if norm else None, q_gamma=gamma, scale=scale)
    qf, of = spread(q.shape, strides, q), spread(q.shape, strides)
    nf.fused_rope_fwd(qf, None, pos, f, q_gamma=gamma, scale=scale, out_q=of)
    assert torch.equal(of, want)
    of.copy_(dq)                             # the gradient, turned back in place
    dg = torch.empty(64, device="cuda") if norm else None
    nf.rope_bwd(of, None, qf if norm else None, None, pos, f, gamma, None, 1e-6, False, False,
                scale, of, None, dg, None)
    assert torch.equal(of, back["dq"])
    if norm:
        assert torch.equal(dg, back["dq_gamma"])


@pytest.mark.parametrize("dtype,N,R,C,G,act", [
    ("f16", 700, 37, 33, 3, "gelu"),         # to 2 bytes
    ("bf16", 520, 75, 66, 6, "silu"),        # to 4
    ("bf16", 500, 21, 36, 4, "gelu"),        # to 8
    ("f32", 610, 19, 33, 1, "silu"),         # to 4
    ("f32", 500, 40, 18, 9, "none"),         # to 8
    ("bf16", 640, 33, 64, 8, "gelu"),        # to 16
])
def test_more_panels_than_clusters(cuda_lib, dtype, N, R, C, G, act):
    """A cluster fetches the next panel's rows while it writes this one's."""
    rng = np.random.default_rng(N + C)
    x, g, b, dy = inputs(rng, dtype, N, R, C)
    check_fwd(cuda_lib, dtype, x, g, b, G, act)
    check_bwd(cuda_lib, dtype, x, g, b, dy, G, act)


def test_calls_at_the_same_time(cuda_lib):
    """Two streams run the operators over and over on their own inputs; every
    result has the bits of the call alone."""
    nf = cuda_lib
    gen = torch.Generator(device="cuda").manual_seed(5)
    new = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()  # noqa: E731
    f, scale = nf.rope_frequencies(64)
    pos = torch.arange(512, device="cuda")
    sets = [(new(2, 9000, 320), new(2, 9000, 320), new(320), new(320), new(2, 512, 8, 64),
             new(64)) for _ in range(2)]

    def run(x, dy, g, b, q, w, stream=None):
        a = nf.fused_group_norm_fwd(x, 32, g, b, activation="silu", stream=stream)
        c = nf.fused_group_norm_bwd(dy, x, 32, g, b, a["mean"], a["rstd"], activation="silu",
                                    stream=stream)
        r = nf.fused_rope_fwd(q, None, pos, f, q_gamma=w, scale=scale, stream=stream)
        s = nf.fused_rope_bwd(r["q"], None, pos, f, q=q, q_gamma=w, scale=scale, stream=stream)
        return a["y"], a["mean"], c["dx"], c["dgamma"], c["dbeta"], r["q"], s["dq"], s["dq_gamma"]

    want = [run(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(sets):
            got[i].append(run(*s, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            for a, c in zip(outs, want[i]):
                assert torch.equal(a, c)
