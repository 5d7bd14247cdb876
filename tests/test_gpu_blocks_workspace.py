"""Workspaces that the caller owns, for every operator that takes one: group
norm forward (two launches) and backward, rotary backward with a norm."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def tensors(gen, *shapes):
    return [torch.randn(s, device="cuda", generator=gen).to(torch.bfloat16) for s in shapes]


class GroupNorm:
    """Forward and backward with a workspace each. 2 x 60000 x 128 takes two
    launches forward; scale multiplies the rows."""

    def __init__(self, nf, seed, scale=1):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        R = 60000 * scale
        self.nf, self.inputs = nf, tensors(gen, (2, R, 128), (2, R, 128), (128,), (128,))

    def __call__(self, wf=None, wb=None):
        x, dy, g, b = self.inputs
        f = self.nf.fused_group_norm_fwd(x, 8, g, b, activation="silu", workspace=wf)
        r = self.nf.fused_group_norm_bwd(dy, x, 8, g, b, f["mean"], f["rstd"], activation="silu",
                                         workspace=wb)
        return [f["y"], f["mean"], f["rstd"], r["dx"], r["dgamma"], r["dbeta"]]


class Rotary:
    """Backward with the heads' norm; scale multiplies the head, which is what
    its workspace grows with."""

    def __init__(self, nf, seed, scale=1):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        D = 64 * scale
        self.nf, self.D = nf, D
        self.inputs = tensors(gen, (2, 900, 8, D), (2, 900, 2, D), (2, 900, 8, D), (2, 900, 2, D),
                              (D,), (D,))
        self.pos = torch.arange(900, device="cuda")
        self.freqs, _ = nf.rope_frequencies(D)

    def __call__(self, _=None, wb=None):
        dq, dk, q, k, gq, gk = self.inputs
        return list(self.nf.fused_rope_bwd(dq, dk, self.pos, self.freqs, q=q, k=k, q_gamma=gq,
                                           k_gamma=gk, workspace=wb).values())


def same(a, b):
    return all(torch.equal(s, t) for s, t in zip(a, b, strict=True))


@pytest.mark.parametrize("op", [GroupNorm, Rotary])
def test_one_workspace_for_call_after_call(cuda_lib, op):
    nf = cuda_lib
    run = op(nf, 1)
    want = run()
    wf, wb = nf.Workspace(), nf.Workspace()
    assert same(run(wf, wb), want)
    assert wb.buf.numel() > 0 and (op is Rotary or wf.buf.numel() > 0)
    at = wf.buf.data_ptr(), wb.buf.data_ptr()
    for w in (wf, wb):
        w.buf.fill_(0x7f)      # what an earlier call left does not matter
    assert same(run(wf, wb), want)
    assert at == (wf.buf.data_ptr(), wb.buf.data_ptr())
    # a tensor of just the bytes that are needed, in a larger buffer
    if op is GroupNorm:
        need = nf.gn_workspace_bytes(2, 60000, 128, 8, torch.bfloat16, True)
    else:
        need = nf.rope_bwd_workspace_bytes(64)
    buf = torch.full((need + 512,), 0x55, dtype=torch.uint8, device="cuda")
    assert same(run(None, buf[256:256 + need]), want)
    assert (buf[:256] == 0x55).all() and (buf[256 + need:] == 0x55).all()
    with pytest.raises(nf.NormError) as e:
        run(None, buf[256:256 + need // 8])
    assert e.value.status == 6


@pytest.mark.parametrize("op", [GroupNorm, Rotary])
def test_a_graph_outlives_the_growth_of_its_workspace(cuda_lib, op):
    nf = cuda_lib
    run, other, large = op(nf, 2), op(nf, 3), op(nf, 4, 4)
    wf, wb = nf.Workspace(), nf.Workspace()
    run(wf, wb)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(wf, wb)
    want, large_want = other(), large()
    assert same(large(wf, wb), large_want)
    assert wb.outgrown, "the larger call did not outgrow the buffer"
    junk = [torch.full_like(b, 0xff) for b in wf.outgrown + wb.outgrown]   # what freed memory might be used for
    for t, v in zip(run.inputs, other.inputs):
        t.copy_(v)
    graph.replay()
    assert same(got, want)
    assert all((j == 0xff).all() for j in junk)
    assert same(large(wf, wb), large_want)


@pytest.mark.parametrize("op", [GroupNorm, Rotary])
def test_two_graphs_at_the_same_time(cuda_lib, op):
    """With a workspace each, replayed on two streams."""
    nf = cuda_lib
    runs = [op(nf, 5), op(nf, 6)]
    want = [r() for r in runs]
    graphs, streams = [], [torch.cuda.Stream() for _ in runs]
    for r in runs:
        ws = nf.Workspace(), nf.Workspace()
        r(*ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = r(*ws)
        graphs.append((g, out, ws))
    torch.cuda.synchronize()
    for _ in range(5):
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, out, _), w in zip(graphs, want):
        assert same(out, w)
