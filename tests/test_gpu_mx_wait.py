"""Failure detection of the product and of the tensor-map transposes without a
fault: their bounded wait, with a short limit, gives up on a barrier at which
nothing arrives, the report is read and cleared, and the context stays usable."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "normalization_fwd_gb300", "csrc")


@pytest.fixture(scope="module")
def helper(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    out = tmp_path_factory.mktemp("wc") / "libwait_cluster.so"
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17", "-shared",
                    "-Xcompiler", "-fPIC", "-I", CSRC, "-o", str(out),
                    os.path.join(ROOT, "tests", "cuda", "wait_cluster.cu")], check=True)
    lib = ctypes.CDLL(str(out))
    lib.wait_cluster_launch.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_longlong, ctypes.c_int]
    return lib


@pytest.mark.gpu
def test_the_wait_gives_up_and_reports(helper, cuda_lib):
    torch.cuda.init()
    gave_up, came = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    cycles = torch.zeros(1, dtype=torch.int64, device="cuda")
    threads, limit = 96, 20_000_000                # some 10 ms
    flags = ctypes.c_uint(0)
    assert helper.wait_cluster_error(ctypes.byref(flags)) == 0 and flags.value == 0
    torch.cuda.synchronize()
    assert helper.wait_cluster_launch(gave_up.data_ptr(), came.data_ptr(), cycles.data_ptr(), limit, threads) == 0
    torch.cuda.synchronize()
    assert int(gave_up) == threads and int(came) == 2 * threads
    # its limit, and less than half a second (a step of the barrier's own waiting) more
    assert limit <= int(cycles) <= limit + 1_000_000_000
    for want in (1, 0):                            # read once, then cleared
        flags = ctypes.c_uint(0)
        assert helper.wait_cluster_error(ctypes.byref(flags)) == 0 and flags.value == want
    nf = cuda_lib
    q = nf.quantize(torch.ones(200, 256, device="cuda"), "mxfp8")
    assert bool((nf.scaled_product(q, q, dtype=torch.float32)["out"] == 256).all())
    assert nf.ln_device_error() == 0


def test_every_source_with_such_waits_is_read():
    """ln_device_error() reads the error word of each translation unit that waits."""
    api = open(os.path.join(CSRC, "api.cu")).read()
    for source, kernels in (("mx.cu", "mx_quantize_kernels.cuh"), ("mx_product.cu", "mx_product_kernels.cuh")):
        assert "g_tu_error" in open(os.path.join(CSRC, kernels)).read()
        text = open(os.path.join(CSRC, source)).read()
        assert f'#include "{kernels}"' in text
        reader = re.search(r"cudaError_t (take_error_\w+)\(.*take_tu_error", text).group(1)
        assert reader in api
