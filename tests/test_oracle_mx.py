"""The oracle of the quantised matrices against torch's own conversions, the
definitions of the formats and facts that hold whatever the rounding."""

import numpy as np
import pytest
import torch

from oracle import mx

RNG = np.random.default_rng(5)


def test_e2m1_values_ties_and_range():
    assert list(mx.round_to_e2m1([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])) == [0, 1, 1, 2, 2, 4, 4]
    assert list(mx.round_to_e2m1([0.2500001, 0.74, -5.1, 7, -100])) == [0.5, 0.5, -6, 6, -6]
    assert list(mx.e2m1_bits([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.5, -6])) == [0, 1, 2, 3, 4, 5, 6, 7, 9, 15]


def test_e4m3_bits_are_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    fine = ~t.isnan()
    assert np.array_equal(mx.e4m3_bits(t[fine].numpy()), np.arange(256)[fine.numpy()])


@pytest.mark.parametrize("most", [448.0, 6.0])
def test_exponent_is_the_least_that_holds(most):
    a = np.concatenate((np.exp(RNG.uniform(-80, 80, 4000)), most * 2.0 ** np.arange(-100.0, 100),
                        np.nextafter(np.float32(most) * np.float32(2.0) ** np.arange(-100, 100).astype(np.float32),
                                     np.float32(np.inf)).astype(float)))
    e = mx.exponent(a, most)
    assert (a <= most * 2.0 ** e.astype(float)).all()
    low = e > -127
    assert (a[low] > most * 2.0 ** (e[low] - 1.0)).all()
    assert mx.exponent(np.zeros(3), most).tolist() == [-127] * 3


@pytest.mark.parametrize("fmt", mx.FORMATS)
def test_values_are_within_half_a_step(fmt):
    v = np.float32(RNG.standard_normal((7, 300)) * np.exp(RNG.uniform(-3, 3, (7, 1)))).astype(float)
    mul = 2688.0 / np.abs(v).max() if fmt == "nvfp4" else None
    mul = None if mul is None else float(np.float32(mul))
    codes, scales, _ = mx.quantize(v, fmt, mul)
    width = mx.BLOCK.get(fmt, 300)
    step = np.repeat(scales, width, axis=1)[:, :300] / (mul or 1.0)
    err = np.abs(mx.values(codes, scales, fmt, mul) - v)
    if fmt in ("mxfp4", "nvfp4"):     # gaps of 1/2 below 2, 1 to 4, 2 to 6
        assert (err <= np.maximum(0.2 * np.abs(v), 0.25 * step) * (1 + 1e-6)).all()
    else:
        assert (err <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * step) * (1 + 1e-6)).all()


def test_blocks_that_are_not_finite():
    v = np.ones((2, 64))
    v[0, 3], v[1, 40] = np.inf, np.nan
    for fmt in mx.FORMATS:
        codes, scales, _ = mx.quantize(v, fmt)
        out = mx.values(codes, scales, fmt)
        width = min(mx.BLOCK.get(fmt, 64), 64)
        bad = np.zeros((2, 64), bool)
        bad[0, :width] = True
        bad[1, 40 // width * width:40 // width * width + width] = True
        assert np.array_equal(np.isnan(out), bad) and (codes[bad] == 0).all()


def test_tiles_have_every_scale_in_its_place():
    s = RNG.integers(1, 255, (200, 11)).astype(np.uint8)
    t = mx.tile(s).reshape(-1)
    assert t.size == 2 * 3 * 512
    for r, b in ((0, 0), (31, 3), (32, 4), (127, 10), (128, 0), (199, 7)):
        at = ((r // 128) * 3 + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4
        assert t[at] == s[r, b]
    assert int((t != 0).sum()) == s.size
