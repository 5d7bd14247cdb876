"""Plain fp64 CPU oracle for rotary positions with the heads' RMSNorm.

TEST INFRASTRUCTURE ONLY: imports nothing from the product package.

Tensors are [batch, tokens, heads, dim] numpy arrays; positions integers
[axes, batch, tokens]; frequencies float64 [axes, pairs] in radians. The
angle is reduced modulo one turn in exact rational arithmetic before its
cosine is taken, so positions of any size are exact.
"""

from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

# 2 pi to 60 digits, as a fraction.
TWO_PI = Fraction("6.28318530717958647692528676655900576839433879875021164194988918")


def angles(positions, freqs):
    """Angles in (-pi, pi], [batch, tokens, pairs]."""
    pos = np.asarray(positions)
    f = [[Fraction(float(v)) / TWO_PI for v in row] for row in np.atleast_2d(freqs)]
    A, B, T = pos.shape
    out = np.empty((B, T, len(f[0])))
    for b in range(B):
        for t in range(T):
            for j in range(len(f[0])):
                turns = sum(int(pos[a, b, t]) * f[a][j] for a in range(A))
                turns -= round(turns)
                out[b, t, j] = float(turns) * 2 * math.pi
    return out


def rotate(u, theta, rot, interleaved, scale, inverse=False):
    """The rotation (or its transpose) of the first ``rot`` elements."""
    out = np.array(u, np.float64)
    c = (np.cos(theta) * scale)[:, :, None, :]
    s = (np.sin(theta) * scale)[:, :, None, :]
    if inverse:
        s = -s
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = np.array(out[..., first]), np.array(out[..., second])
    out[..., first] = a * c - b * s
    out[..., second] = b * c + a * s
    return out


def _weight(gamma, zero_centered):
    g = np.asarray(gamma, np.float64)
    return 1.0 + g if zero_centered else g


def rope_fwd(x, theta, rot, *, gamma=None, eps=0.0, interleaved=False, scale=1.0,
             zero_centered=False) -> dict:
    u = np.asarray(x, np.float64)
    if gamma is not None:
        rstd = 1.0 / np.sqrt((u * u).mean(axis=-1, keepdims=True) + eps)
        u = u * rstd * _weight(gamma, zero_centered)
    return {"y": rotate(u, theta, rot, interleaved, scale), "u": u}


def rope_bwd(dy, x, theta, rot, *, gamma=None, eps=0.0, interleaved=False, scale=1.0,
             zero_centered=False) -> dict:
    g = rotate(dy, theta, rot, interleaved, scale, inverse=True)
    if gamma is None:
        return {"dx": g, "dgamma": None}
    x = np.asarray(x, np.float64)
    rstd = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    xhat = x * rstd
    out = {"dgamma": (g * xhat).sum(axis=(0, 1, 2)),
           "dgamma_abs": np.abs(g * xhat).sum(axis=(0, 1, 2))}
    g = g * _weight(gamma, zero_centered)
    c = (g * xhat).mean(axis=-1, keepdims=True)
    out["dx"] = rstd * (g - xhat * c)
    # the size of the terms that dx is made of, for the tests' bounds
    out["dx_terms"] = rstd * (np.abs(g) + np.abs(xhat) * np.abs(g * xhat).mean(-1, keepdims=True))
    return out
