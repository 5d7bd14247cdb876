"""A row's result does not depend on how many rows the call has, although few
rows are spread over more threads than many."""

import pytest
import torch

from _mx import DT, FORMATS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ["layernorm", "rmsnorm"])
@pytest.mark.parametrize("dtype,rows,hidden", [
    ("bf16", 400, 8192), ("bf16", 700, 5120), ("f16", 6000, 320), ("bf16", 5000, 520), ("f32", 1200, 1000),
    ("f32", 300, 8192), ("bf16", 2000, 1160), ("f16", 250, 16384), ("f32", 20000, 32), ("bf16", 9000, 256),
    ("f32", 500, 2600), ("f16", 300, 12296), ("bf16", 300, 1165),
    ("bf16", 3000, 1280), ("bf16", 300, 4096)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_alone_are_the_same_rows(cuda_lib, fmt, dtype, rows, hidden, mode):
    nf = cuda_lib
    gen = torch.Generator(device="cuda").manual_seed(hidden)

    def t(*shape, std=1.0, mean=0.0):
        return (mean + std * torch.randn(shape, generator=gen, device="cuda")).to(DT[dtype])

    x, r = t(rows, hidden, mean=0.3), t(rows, hidden)
    g, b = t(hidden, std=0.2, mean=1.0), t(hidden, std=0.2)
    kw = dict(format=fmt, mode=mode, store_y=True)
    whole = nf.fused_norm_quant_fwd(x, g, b, residual=r, **kw)
    values = nf.dequantize(whole["q"])
    names = ["sum", "y", "rstd"] + (["mean"] if mode == "layernorm" else [])
    for n in (1, 40):
        for at in range(0, min(rows, 5 * n), n) if n == 1 else range(0, min(rows, 400), n):
            part = nf.fused_norm_quant_fwd(x[at:at + n], g, b, residual=r[at:at + n], **kw)
            for k in names:
                assert torch.equal(part[k], whole[k][at:at + n]), (k, at)
            assert torch.equal(part["q"].codes.view(torch.uint8), whole["q"].codes.view(torch.uint8)[at:at + n])
            assert torch.equal(nf.dequantize(part["q"]), values[at:at + n])
