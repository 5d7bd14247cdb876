"""Helpers of the group norm and rotary position tests: padded buffers that
show writes outside of a tensor, strided views, half steps of the formats."""

from __future__ import annotations

import numpy as np
import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24                      # half a step of fp32, relative
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}   # least positive value


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def make(rng, shape, dtype, std=1.0, mean=0.0):
    """A CPU tensor of mean + std * N(0, 1), rounded to dtype."""
    a = mean + std * rng.standard_normal(shape)
    return torch.from_numpy(np.asarray(a, np.float32)).to(DTYPES[dtype])


class Padded:
    """A CUDA tensor `t` of `shape` inside a larger buffer: `extra` more
    columns in its last dimension (they make it strided) and a margin at
    either end. intact() says whether all of that still has its fill."""

    def __init__(self, shape, dtype, extra=0, offset=0, fill=7.0, data=None):
        wide = tuple(shape[:-1]) + (shape[-1] + extra,)
        n = int(np.prod(wide))
        self.margin = 64
        self.buf = torch.full((self.margin + offset + n + self.margin,), fill, dtype=dtype,
                              device="cuda")
        at = self.margin + offset
        self.t = self.buf[at:at + n].view(wide)[..., :shape[-1]]
        self.fill = fill
        self.mask = torch.ones_like(self.buf, dtype=torch.bool)
        self.mask[at:at + n].view(wide)[..., :shape[-1]] = False
        if data is not None:
            self.t.copy_(data)

    def intact(self):
        return bool((self.buf[self.mask] == self.fill).all())


def within(got, want, tol, what):
    """Every element within its bound; where `want` is not finite, equal."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    tol = np.broadcast_to(tol, want.shape)
    assert got.shape == want.shape, f"{what}: {got.shape} for {want.shape}"
    odd = ~np.isfinite(want)
    assert np.array_equal(got[odd], want[odd], equal_nan=True), f"{what}: not the same inf or NaN"
    err, bound = np.abs(got - want)[~odd], tol[~odd]
    if not err.size:
        return 0.0
    assert np.isfinite(err).all(), f"{what}: {int((~np.isfinite(err)).sum())} values not finite"
    worst = float(np.max(err / np.maximum(bound, 1e-300)))
    assert worst <= 1.0, f"{what}: error up to {worst:.3g} times the bound"
    return worst
