"""Which library the binding's calls reach, and that they do without its C++ part."""

import os
import shutil
import subprocess
import sys

import pytest

import normalization_fwd_gb300 as nf

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def built():
    return nf.build_library()


def child(code, *args):
    r = subprocess.run([sys.executable, "-c", code, *args], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_a_library_elsewhere_is_the_only_one(built, tmp_path):
    """With a path of the caller's own, the C++ part calls that library too: no
    other copy of it, with error words and settings of its own, is in the process."""
    other = str(tmp_path / "elsewhere.so")
    shutil.copy(built, other)
    out = child(
        "import sys, normalization_fwd_gb300 as nf\n"
        "nf.load_library(sys.argv[1])\n"
        "assert nf._marshal is not None\n"
        "print(nf.mx_matrix_bytes('mxfp8', 3, 40))\n"
        "print(sorted({l.split()[-1] for l in open('/proc/self/maps') if l.rstrip().endswith('.so')}))\n", other)
    assert "(192, 512)" in out and other in out and built not in out


def test_without_the_cpp_part(built, tmp_path):
    """A library built under another torch serves this one."""
    out = child(
        "import normalization_fwd_gb300 as nf, sys\n"
        "nf.marshal_path = lambda: sys.argv[1]\n"
        "nf.load_library()\n"
        "print(nf._marshal, nf.mx_matrix_bytes('nvfp4', 3, 40), nf.ln_status_string(0))\n",
        str(tmp_path / "none.so"))
    assert out.startswith("None (96, 512)")


CALLS = ("fused_norm_quant_fwd", "quantize", "dequantize", "scaled_product", "fused_norm_fwd_from_partials")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_both_ways_give_the_same(cuda_lib, monkeypatch, fmt):
    import torch
    x, r = (torch.randn(70, 320, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w, g = torch.randn(90, 320, device="cuda"), torch.ones(320, device="cuda", dtype=torch.bfloat16)
    h = torch.ones(90, device="cuda", dtype=torch.bfloat16)

    def run():
        f = cuda_lib.fused_norm_quant_fwd(x, g, format=fmt, residual=r, mode="rmsnorm")
        p = cuda_lib.scaled_product(f["q"], cuda_lib.quantize(w, fmt), partials=True)
        z = cuda_lib.fused_norm_fwd_from_partials(p["out"], p["psum"], p["psq"], p["tile_cols"], h, h, kind="sum_m2")
        return f["sum"], cuda_lib.dequantize(f["q"]), p["out"], p["psum"], z["y"], z["mean"]

    assert cuda_lib._marshal is not None
    calls = []

    class Counted:
        def __getattr__(self, name):
            calls.append(name)
            return getattr(marshal, name)

    marshal = cuda_lib._marshal
    monkeypatch.setattr(cuda_lib, "_marshal", Counted())
    want = run()
    assert len(calls) == len(CALLS)                # the C++ part is what ran
    monkeypatch.setattr(cuda_lib, "_marshal", None)
    for a, b in zip(run(), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("lacking", ["g++", "a torch with CUDA", "torch's headers", "nothing"])
def test_the_library_builds_without_what_only_the_cpp_part_wants(built, monkeypatch, tmp_path, lacking):
    """The commands of a build, none of them run."""
    import torch

    from normalization_fwd_gb300 import build as b
    ran, moved = [], []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        ran.append(cmd)
        return Done

    which = shutil.which
    if lacking == "g++":
        monkeypatch.setattr(b.shutil, "which", lambda name, *a, **k: None if name == "g++" else which(name, *a, **k))
    elif lacking == "a torch with CUDA":
        monkeypatch.setattr(torch.version, "cuda", None)
    elif lacking == "torch's headers":
        monkeypatch.setattr(torch, "__file__", str(tmp_path / "torch" / "__init__.py"))
    # the library alone, newer than its sources
    with monkeypatch.context() as m:
        made = tmp_path / "lib.so"
        made.touch()
        m.setattr(b, "LIB_PATH", str(made))
        m.setattr(b, "marshal_path", lambda: str(tmp_path / "none.so"))
        assert b.up_to_date() == (lacking != "nothing")
    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b.os, "replace", lambda src, dst: moved.append(dst))
    assert b.build(force=True) == b.LIB_PATH
    host = [c for c in ran if c[0] == "g++"]
    assert len(host) == (2 if lacking == "nothing" else 0)
    assert len(ran) == len(b._sources()) + 1 + len(host)
    assert moved == [b.LIB_PATH] + ([b.marshal_path()] if host else [])


def test_an_unknown_kind_of_partials(built):
    """The binding's own error, whichever way the call would go."""
    import torch
    x = torch.zeros(2, 64)
    p = torch.zeros(2, 1)
    with pytest.raises(ValueError, match="unknown partial kind 'sum'"):
        nf.fused_norm_fwd_from_partials(x, p, p, 64, x[0], kind="sum")


@pytest.mark.gpu
def test_an_unknown_kind_of_partials_on_the_gpu(cuda_lib):
    import torch
    x, p = torch.zeros(2, 64, device="cuda"), torch.zeros(2, 1, device="cuda")
    for kw in ({}, {"stream": torch.cuda.current_stream()}, {"amax": True}):
        with pytest.raises(ValueError, match="unknown partial kind 'sum'"):
            cuda_lib.fused_norm_fwd_from_partials(x, p, p, 64, x[0], kind="sum", **kw)


def test_a_cpp_part_of_another_state_is_not_taken(built, monkeypatch, tmp_path):
    """One that was built from other declarations than the library's, under another
    torch say, has another name."""
    from normalization_fwd_gb300 import build as b
    now = b.marshal_path()
    assert os.path.isfile(now)
    for path in ("include/normfuse.h", "normalization_fwd_gb300/csrc/marshal.cc"):
        target = tmp_path / path
        target.parent.mkdir(parents=True, exist_ok=True)
        shutil.copy(os.path.join(ROOT, path), target)
    monkeypatch.setattr(b, "ROOT", str(tmp_path))
    monkeypatch.setattr(b, "CSRC", str(tmp_path / "normalization_fwd_gb300" / "csrc"))
    assert b.marshal_path() == now
    for path in ("include/normfuse.h", "normalization_fwd_gb300/csrc/marshal.cc"):
        with open(tmp_path / path, "a") as f:
            f.write("// another state\n")
        assert b.marshal_path() != now
        now = b.marshal_path()
