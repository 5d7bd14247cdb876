import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_addoption(parser):
    parser.addoption(
        "--ring-kernels", default="",
        help="comma-separated directions (forward, backward, softmax) whose calls the GPU "
             "tests plan with the bulk-copy ring kernels instead of the default ones "
             "(through the library's testing hook ln_testing_select_kernels)")


def pytest_configure(config):
    config.addinivalue_line(
        "markers", "gpu: needs a CUDA GPU (sm_103a); runs the CUDA library through its C ABI")


# Tests without a GPU mark whose calls the C library accepts, on addresses that
# are no memory: they end at the missing device, and would launch on one.
MADE_UP_ADDRESSES = ("test_gn_fwd_slices_of_one_buffer", "test_rope_overlap_of_packed_heads")


def pytest_collection_modifyitems(items):
    import torch
    if not torch.cuda.is_available():
        return
    for item in items:
        if getattr(item, "originalname", None) in MADE_UP_ADDRESSES:
            item.add_marker(pytest.mark.skip(
                reason="a GPU is visible: the call would be launched on made-up addresses"))


@pytest.fixture(scope="session")
def cuda_lib(request):
    """The CUDA library, built in-tree; the GPU tests fail loudly without it."""
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU test selected but no CUDA device is visible")
    import normalization_fwd_gb300 as nf
    nf.load_library()
    ring = {d for d in request.config.getoption("--ring-kernels").split(",") if d}
    unknown = ring - {"forward", "backward", "softmax"}
    if unknown:
        pytest.fail(f"--ring-kernels: unknown direction(s) {sorted(unknown)}")
    fam = {d: ("ring" if d in ring else "default") for d in ("forward", "backward", "softmax")}
    nf.ln_testing_select_kernels(**fam)
    return nf
