"""What the sources of the quantised operators' kernels have to keep to, read
from the sources: these are rules whose breach no run shows reliably (a race, an
order that only another library's kernel would break)."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "normalization_fwd_gb300", "csrc")


def code(path):
    """A source without its comments."""
    text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


SOURCES = {os.path.basename(p): code(p) for p in sorted(glob.glob(os.path.join(CSRC, "mx_*.cuh"))
                                                        + glob.glob(os.path.join(CSRC, "tcgen05.cuh")))}


def kernels(text):
    """name -> body of the kernels in a source."""
    out = {}
    for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\s*\(", text):
        start = text.index("{", m.end())
        depth, i = 0, start
        while True:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
            if depth == 0:
                break
        out[m.group(1)] = text[start:i]
    return out


KERNELS = {name: body for text in SOURCES.values() for name, body in kernels(text).items()}


def test_kernels_are_found():
    assert {"mx_norm_tile_kernel", "mx_norm_cta_kernel", "mx_norm_ragged_kernel", "quant_block_kernel",
            "quant_row_kernel", "quant_transpose_kernel", "quant_transpose_tma_kernel",
            "quant_transpose_row_tma_kernel", "dequant_kernel", "product_tile_kernel",
            "product_pair_kernel"} == set(KERNELS)


@pytest.mark.parametrize("name", sorted(SOURCES))
def test_no_load_that_wants_memory_constant(name):
    """These kernels may be resident while the one in front of them on the
    stream still writes, so nothing that they read is constant for as long as
    they live: no non-coherent load, and no pointer that lets the compiler
    make one."""
    found = re.findall(r"__ldg|\bld_vec\w*|ld\.global(?:\.\w+)*\.nc\b|__restrict__|__ldcs\b", SOURCES[name])
    assert not found


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_tensor_memory_is_taken_between_the_wait_and_the_signal(name):
    """A kernel that held tensor memory while it waits for the one in front, or
    let the next one start before it has its own, could wait for columns that
    a kernel holds which waits for it."""
    body = KERNELS[name]
    if "tmem_alloc" not in body:
        assert body.count("start_after_stream()") == 1
        return
    steps = ["wait_for_stream()", "tmem_alloc", "__syncthreads()", "let_next_start()"]
    at = [body.index(s) for s in steps]
    assert at == sorted(at) and "start_after_stream" not in body
    assert all(body.count(s) == 1 for s in (steps[0], steps[1], steps[3]))


def test_looking_ahead_does_not_hold_work_back():
    """A product's issuing warp asks for the next stage before it issues the work of
    this one: by a test that returns at once, and only for a stage that will come."""
    text = SOURCES["mx_product_kernels.cuh"]
    asked = [a for a in re.findall(r"\bhere\s*=\s*([^;]*);", text) if "mbar_wait_cluster" not in a]
    assert len(asked) == 4 and all("mbar_ready_cluster" in a for a in asked)
    assert all("smem_addr(&full[0])" in a or re.match(r"\(?c \+ 1 <", a) for a in asked)
    assert "mbar_test_cluster" not in text
    body = re.search(r"bool mbar_ready_cluster\(.*?\n}", SOURCES["tcgen05.cuh"], flags=re.S).group(0)
    assert "mbarrier.test_wait" in body and "try_wait" not in body
