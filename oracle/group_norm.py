"""Plain fp64 CPU oracle for the group norm with an activation, channels last.

TEST INFRASTRUCTURE ONLY: imports nothing from the product package.

``x`` is [samples, rows, channels]; group g has the channels
[g, g + 1) * channels / groups. gamma and beta are [channels],
[samples, channels] or None. Everything runs in float64; nothing is rounded.
"""

from __future__ import annotations

import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def normal_cdf(z):
    return 0.5 * _erfc(-np.asarray(z, np.float64) / math.sqrt(2.0))


def activate(z, act):
    """(act(z), act'(z)) for "none", "silu" or "gelu"."""
    if act == "none":
        return z, np.ones_like(z)
    if act == "silu":
        with np.errstate(over="ignore"):
            s = np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))),
                         np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
        return z * s, s + z * s * (1 - s)
    if act == "gelu":
        p = normal_cdf(z)
        return z * p, p + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    raise ValueError(f"unknown activation {act!r}")


def _weights(p, zero_centered, shape, default):
    """gamma or beta as [samples, 1, channels]."""
    N, _, C = shape
    if p is None:
        return np.full((N, 1, C), default)
    p = np.broadcast_to(np.asarray(p, np.float64), (N, C)).reshape(N, 1, C)
    return p + 1.0 if zero_centered else p


def _spread(t, C):
    """[samples, groups] -> [samples, 1, channels]."""
    return np.repeat(t, C // t.shape[1], axis=1)[:, None, :]


def _group_mean(t, groups):
    """Mean over rows and the group's channels: [samples, groups]."""
    N, R, C = t.shape
    return t.reshape(N, R, groups, C // groups).mean(axis=(1, 3))


def group_norm_fwd(x, groups, gamma, beta, eps, act="none", zero_centered=False) -> dict:
    x = np.asarray(x, np.float64)
    C = x.shape[2]
    w = _weights(gamma, zero_centered, x.shape, 1.0)
    b = _weights(beta, False, x.shape, 0.0)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        mean = _group_mean(x, groups)
        d = x - _spread(mean, C)
        rstd = 1.0 / np.sqrt(_group_mean(d * d, groups) + eps)
        z = d * _spread(rstd, C) * w + b
        return {"y": activate(z, act)[0], "z": z, "mean": mean, "rstd": rstd, "w": w, "b": b}


def group_norm_bwd(dy, x, groups, gamma, beta, mean, rstd, act="none", zero_centered=False) -> dict:
    """dx, and the per-sample column sums dgamma, dbeta [samples, channels]
    (their sum over the samples is the gradient of shared parameters)."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    C = x.shape[2]
    w = _weights(gamma, zero_centered, x.shape, 1.0)
    b = _weights(beta, False, x.shape, 0.0)
    rs = _spread(np.asarray(rstd, np.float64), C)
    xhat = (x - _spread(np.asarray(mean, np.float64), C)) * rs
    dz = dy * activate(xhat * w + b, act)[1]
    g = w * dz
    c1, c2 = _group_mean(g, groups), _group_mean(g * xhat, groups)
    dx = rs * (g - _spread(c1, C) - xhat * _spread(c2, C))
    return {"dx": dx, "dgamma": (dz * xhat).sum(axis=1), "dbeta": dz.sum(axis=1), "xhat": xhat,
            "dz": dz, "w": w}
