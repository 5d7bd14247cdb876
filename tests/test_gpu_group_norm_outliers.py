"""Group norm statistics of data whose first rows say nothing about the rest:
an outlier, padding of zeros under a large mean, a step.

Bounds, with u = 2^-24. A thread sums a column over blocks of 8, 24 and then 32
of its rows, each block about the mean of the rows before it (the first about
its first row). The first block's squares come to at most 8 M2, all the later
ones' to at most 4 M2 (Cauchy: with b rows of N, s1^2 / N <= s2 b / N, b / N <= 3 / 4).

* M2 of a thread: a square's difference is rounded (2 u), a block adds up to 8 or
  32 of them one after the other, the move costs a few roundings a block, and
  there are at most 20 blocks (512 rows): 8 * 10 u, 4 * 34 u and 20 u, 236 u.
* Merges over at most 256 lanes in parts, 2048 columns and parts of a group
  dealt to 32 lanes and 512 slices dealt to 32 lanes: 64 additions and some 20
  products and quotients. In all 320 u of var, half of it and 4 u of rstd: 164 u.
* mean: a block's sum of differences d costs 32 u of the sum of their sizes. What
  a single value x adds to those sizes, as itself and in the means that it
  draws along (8 and 24 rows, then 32 at a time of a growing number: 7 + 3 + 1
  + 1 / 2 + 1 / 3 ...), is at most 16 |x - mean|: 512 u of mean|x - mean|, and
  4 u of |mean| for the roundings of the means themselves.
* y: the mean's error times rstd |w|, the relative error of rstd times the term
  that it scales, 4 u of either term and the output's half step.
"""

import pytest
import torch

from _blocks import DTYPES, HALF, U

pytestmark = pytest.mark.gpu

# (dtype, samples, rows, channels, groups); most rows a thread adds up, in brackets
SHAPES = [
    ("f32", 228, 16384, 32, 4),        # a CTA a panel (512)
    ("f32", 29, 16384, 128, 8),        # two CTAs a panel (256)
    ("f32", 228, 65536, 8, 2),         # two vectors a row, one CTA (512)
    ("bf16", 34, 262144, 8, 1),        # one vector a row, two launches (40)
    ("f32", 3, 5000, 96, 3),           # clusters of small panels
    ("f32", 2, 20000, 1024, 1),        # groups over many tiles
    ("f16", 2, 3001, 33, 3),           # rows aligned to 2 bytes
]


def pattern(x, kind):
    """Rows that are not like the others, in place; x is N(0, 1)."""
    R = x.shape[1]
    if kind.startswith("first"):
        x[:, 0] = float(kind[5:])
    elif kind == "zero under 100":
        x += 100
        x[:, 0] = 0
    elif kind == "padding":
        x += 100
        x[:, :R // 14] = 0
    elif kind == "middle":
        x[:, R // 2 + 1] = 3000
    elif kind == "step":
        x[:, R // 2:] += 50


@pytest.mark.parametrize("dtype,N,R,C,G", SHAPES)
@pytest.mark.parametrize("kind", ["first1000", "first10000", "zero under 100", "padding", "middle",
                                  "step"])
def test_statistics(cuda_lib, dtype, N, R, C, G, kind):
    gen = torch.Generator(device="cuda").manual_seed(R + C)
    x = torch.randn(N, R, C, device="cuda", generator=gen)
    pattern(x, kind)
    x = x.to(DTYPES[dtype])
    w, b = (torch.randn(C, device="cuda", generator=gen).to(DTYPES[dtype]) for _ in range(2))
    f = cuda_lib.fused_group_norm_fwd(x, G, w, b)
    worst = 0.0
    for n in range(0, N, max(1, N // 16)):
        xr = x[n].double().view(R, G, C // G)
        m = xr.mean((0, 2))
        d = xr - m[:, None]
        rs = (d.square().mean((0, 2)) + 1e-5).rsqrt()
        tol_m = 512 * U * d.abs().mean((0, 2)) + 4 * U * m.abs()
        tol_r = 164 * U * rs
        em, er = (f["mean"][n].double() - m).abs(), (f["rstd"][n].double() - rs).abs()
        worst = max(worst, float((er / rs).max()))
        assert (em <= tol_m).all(), f"mean: {float((em / tol_m).max()):.3g} times the bound"
        assert (er <= tol_r).all(), f"rstd: {float((er / tol_r).max()):.3g} times the bound"
        wg, bg = w.double().view(G, -1), b.double().view(G, -1)
        term = d * rs[:, None] * wg
        y = term + bg
        tol = ((tol_m * rs)[:, None] * wg.abs() + (164 + 4) * U * term.abs() + 4 * U * bg.abs()
               + HALF[dtype] * y.abs() + 2.0 ** -24)
        assert ((f["y"][n].double().view_as(y) - y).abs() <= tol).all()
    print(f"rstd off by {worst / U:.1f} u at most")
