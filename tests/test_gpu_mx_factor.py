"""The product's factor, alpha over both operands' mul, where it or a part of it
is no fp32 number and the results are."""

import numpy as np
import pytest
import torch

from _blocks import U, f64, within
from _mx import device_matrix, exact_operand, on_gpu
from oracle import mx

pytestmark = pytest.mark.gpu

# alpha, mul of A, mul of B
FACTORS = [
    (1.0, 7.3e21, 6.9e21),        # 2e-44, a subnormal: results of 1e-41 and, with large sums, more
    (3.0e4, 7.3e21, 6.9e21),
    (1.0e12, 1.3e30, 2.7e20),     # the quotient by the first alone is 1e-18
    (100.0, 1.0e-38, 3.0e38),     # the quotient by the first is past the largest number
    (1.0e-30, 2.0e30, 1.0e-38),   # and here far below the least
    (-7.0e-3, 1.0e-20, 3.0e-20),  # sums of 0 have results of 0, others past the range
    (1.0, 1.2e-38, 1.1e-38),
    (2.0, 3.0e38, 2.0e38),        # all results are 0
    (1.0e-40, 1.0e-25, 1.0e-20),  # a subnormal alpha
    (0.0, 1.0e-30, 1.0e-30),
    (1.5, 96.0, 28.0),
]


@pytest.mark.parametrize("M,N,K", [(5, 300, 320), (140, 257, 320), (2600, 2000, 96), (2560, 4096, 64)])
@pytest.mark.parametrize("alpha,ma,mb", FACTORS)
def test_results_are_those_of_the_quotient(cuda_lib, M, N, K, alpha, ma, mb):
    nf = cuda_lib
    rng = np.random.default_rng(M)
    (ac, as_), (bc, bs) = exact_operand(rng, M, K, "nvfp4"), exact_operand(rng, N, K, "nvfp4")
    ac[1] = 0.0
    bc[3] = 0.0
    alpha, ma, mb = (float(np.float32(v)) for v in (alpha, ma, mb))
    a, b = device_matrix(nf, ac, as_, "nvfp4", on_gpu(ma)), device_matrix(nf, bc, bs, "nvfp4", on_gpu(mb))
    sums, size = mx.product(mx.values(ac, as_, "nvfp4"), mx.values(bc, bs, "nvfp4"))
    assert size.max() < 2 ** 19            # the sums are exact
    want = sums * alpha / ma / mb
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    # two quotients, two products: a rounding each, and of a subnormal result two
    # roundings to multiples of 2^-149
    for res in (None, torch.zeros(M, N, device="cuda")):
        got = f64(nf.scaled_product(a, b, alpha=alpha, residual=res, dtype=torch.float32)["out"])
        within(got, want, 4.1 * U * np.abs(want) + 2.0 ** -149, "out")
    assert not np.isnan(got).any() and (got[1] == 0).all() and (got[:, 3] == 0).all()
    assert nf.ln_device_error() == 0
