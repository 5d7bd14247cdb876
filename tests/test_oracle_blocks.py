"""Pins of the group norm and rotary position oracles: invariants, central
differences, and what the rotation is as a complex product."""

import numpy as np
import pytest

from oracle import group_norm_bwd, group_norm_fwd, rope_angles, rope_bwd, rope_fwd
from oracle.group_norm import activate, normal_cdf

EPS = 1e-5


def gn_case(act, per_sample, zero_centered, seed=0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((2, 5, 6)) * 1.5 + 0.7
    shape = (2, 6) if per_sample else (6,)
    return x, rng.standard_normal(shape), rng.standard_normal(shape), rng.standard_normal(x.shape)


def test_normal_cdf_and_activations():
    assert normal_cdf(0.0) == 0.5
    assert abs(float(normal_cdf(1.0)) - 0.8413447460685429) < 1e-15
    assert abs(float(normal_cdf(-8.0)) / 6.220960574271785e-16 - 1) < 1e-12
    z = np.array([-1000.0, -3.0, 0.0, 2.0, 1000.0])
    silu, _ = activate(z, "silu")
    assert silu[0] == 0 and silu[2] == 0 and silu[4] == 1000.0
    assert abs(silu[3] - 2 / (1 + np.exp(-2.0))) < 1e-15
    for act in ("silu", "gelu"):
        h = 1e-6
        num = (activate(z[1:4] + h, act)[0] - activate(z[1:4] - h, act)[0]) / (2 * h)
        assert np.allclose(num, activate(z[1:4], act)[1], atol=1e-9)
    with pytest.raises(ValueError):
        activate(z, "relu")


def test_group_norm_invariants():
    x, _, _, _ = gn_case("none", False, False)
    y = group_norm_fwd(x, 3, None, None, 0.0)["y"].reshape(2, 5, 3, 2)
    assert np.allclose(y.mean(axis=(1, 3)), 0, atol=1e-14)
    assert np.allclose(y.var(axis=(1, 3)), 1, atol=1e-13)
    # one group a channel and one group in all, by hand
    y = group_norm_fwd(x, 6, None, None, 0.0)["y"]
    assert np.allclose(y, (x - x.mean(1, keepdims=True)) / x.std(1, keepdims=True))
    y = group_norm_fwd(x, 1, None, None, 0.0)["y"]
    assert np.allclose(y[1], (x[1] - x[1].mean()) / x[1].std())


def test_group_norm_groups_do_not_meet():
    x, g, b, _ = gn_case("silu", False, False)
    want = group_norm_fwd(x, 3, g, b, EPS, "silu")["y"]
    x[1, 2, 3] = np.nan
    got = group_norm_fwd(x, 3, g, b, EPS, "silu")["y"]
    assert np.isnan(got[1, :, 2:4]).all()
    assert np.array_equal(got[0], want[0])
    assert np.array_equal(got[1, :, :2], want[1, :, :2])


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("per_sample,zero_centered", [(False, False), (True, True)])
def test_group_norm_gradients_match_differences(act, per_sample, zero_centered):
    x, gamma, beta, dy = gn_case(act, per_sample, zero_centered)

    def loss(x, gamma, beta):
        return float((group_norm_fwd(x, 2, gamma, beta, EPS, act, zero_centered)["y"] * dy).sum())

    f = group_norm_fwd(x, 2, gamma, beta, EPS, act, zero_centered)
    b = group_norm_bwd(dy, x, 2, gamma, beta, f["mean"], f["rstd"], act, zero_centered)
    grads = [b["dx"], b["dgamma"] if per_sample else b["dgamma"].sum(0),
             b["dbeta"] if per_sample else b["dbeta"].sum(0)]
    h = 1e-6
    for i, got in enumerate(grads):
        args = [x, gamma, beta]
        num = np.empty_like(args[i])
        for at in np.ndindex(args[i].shape):
            up, down = [a.copy() for a in args], [a.copy() for a in args]
            up[i][at] += h
            down[i][at] -= h
            num[at] = (loss(*up) - loss(*down)) / (2 * h)
        assert np.allclose(num, got, atol=2e-8), i


def test_a_group_of_one_value_has_no_gradient():
    rng = np.random.default_rng(3)
    x, dy = rng.standard_normal((2, 1, 4)), rng.standard_normal((2, 1, 4))
    f = group_norm_fwd(x, 4, None, None, EPS, "silu")
    assert np.array_equal(f["mean"], x[:, 0])
    b = group_norm_bwd(dy, x, 4, None, None, f["mean"], f["rstd"], "silu")
    assert (b["dx"] == 0).all()


def test_angles_are_exact_far_out():
    f = np.array([[1.0, 0.25, 1e-4]])
    got = rope_angles(np.array([[[0, 1, -1, 10 ** 9]]]), f)
    assert (got[0, 0] == 0).all()
    assert np.allclose(got[0, 1], [1.0, 0.25, 1e-4], rtol=1e-14)
    assert np.allclose(got[0, 2], -got[0, 1], rtol=1e-14)
    # cos(10^9), cos(2.5 * 10^8) and cos(10^5) from tables
    assert np.allclose(np.cos(got[0, 3]), [0.83788718136390, np.cos(2.5e8), np.cos(1e5)], atol=1e-10)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 3, 2, 10))
    th = rng.uniform(-3, 3, (2, 3, 4))
    y = rope_fwd(x, th, 8, interleaved=interleaved, scale=1.25)["y"]
    a, b = (x[..., 0:8:2], x[..., 1:8:2]) if interleaved else (x[..., :4], x[..., 4:8])
    z = (a + 1j * b) * 1.25 * np.exp(1j * th)[:, :, None]
    got = (y[..., 0:8:2] + 1j * y[..., 1:8:2]) if interleaved else y[..., :4] + 1j * y[..., 4:8]
    assert np.allclose(z, got, atol=1e-14)
    assert np.array_equal(y[..., 8:], x[..., 8:])


def test_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 1, 16))
    f = 100.0 ** (-np.arange(8) / 8)[None]
    def score(m, n):
        a = rope_fwd(q, rope_angles(np.array([[[m]]]), f), 16)["y"]
        return float((a * rope_fwd(k, rope_angles(np.array([[[n]]]), f), 16)["y"]).sum())
    assert abs(score(5, 3) - score(1002, 1000)) < 1e-12


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradients_match_differences(norm, interleaved):
    rng = np.random.default_rng(4)
    x, dy = rng.standard_normal((2, 1, 3, 2, 6))
    th = rng.uniform(-3, 3, (1, 3, 2))
    gamma = rng.standard_normal(6) if norm else None
    kw = dict(eps=1e-3, interleaved=interleaved, scale=0.8, zero_centered=True)
    b = rope_bwd(dy, x, th, 4, gamma=gamma, **kw)
    h = 1e-6
    num = np.empty_like(x)
    for at in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[at] += h
        down[at] -= h
        num[at] = ((rope_fwd(up, th, 4, gamma=gamma, **kw)["y"]
                    - rope_fwd(down, th, 4, gamma=gamma, **kw)["y"]) * dy).sum() / (2 * h)
    assert np.allclose(num, b["dx"], atol=2e-8)
    if norm:
        num = np.empty(6)
        for i in range(6):
            e = np.eye(6)[i] * h
            num[i] = ((rope_fwd(x, th, 4, gamma=gamma + e, **kw)["y"]
                       - rope_fwd(x, th, 4, gamma=gamma - e, **kw)["y"]) * dy).sum() / (2 * h)
        assert np.allclose(num, b["dgamma"], atol=2e-8)
