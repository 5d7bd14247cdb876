"""The group norm's and rotary positions' C entry points over a device that is
not there (tests/cuda/fake_device.cc): built from the library's own gn.cu and
rope.cu, loaded beside the library."""

from __future__ import annotations

import ctypes
import os
import subprocess

import normalization_fwd_gb300 as nf
from normalization_fwd_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
COUNTS = ("launches", "grid", "cluster", "finalizes", "memsets")


def load(folder):
    """Build the library into `folder` and load it."""
    out = os.path.join(str(folder), "libfake_device.so")
    sources = [os.path.join(ROOT, "tests", "cuda", "fake_device.cc"),
               os.path.join(build.CSRC, "gn.cu"), os.path.join(build.CSRC, "rope.cu")]
    # -Bsymbolic: its own definitions, whatever the process has loaded besides
    subprocess.run([build.find_nvcc(), *build.ARCH, "-O1", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-shared", "-cudart", "none", "-Xlinker", "-Bsymbolic", "-o", out, *sources],
                   check=True)
    lib = ctypes.CDLL(out)
    for name in nf.exported_symbols("gn_") + nf.exported_symbols("rope_"):
        getattr(lib, name).argtypes = getattr(nf.load_library(), name).argtypes
        getattr(lib, name).restype = ctypes.c_int
    return lib


def reset(lib, sms=152, most_cluster=16):
    """A device of so many SMs that places clusters of so many CTAs."""
    lib.fake_reset(sms, most_cluster)


def counts(lib):
    """What was launched since the last reset."""
    out = (ctypes.c_int * len(COUNTS))()
    lib.fake_counts(out)
    return dict(zip(COUNTS, out))
