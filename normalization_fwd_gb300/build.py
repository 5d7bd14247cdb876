"""Build the CUDA library ``libnormfuse.so`` in-tree for sm_103a, and the
binding's C++ part beside it.

Each ``csrc/*.cu`` translation unit is compiled by nvcc in parallel, then the
objects are linked into a shared library next to this file (the CUDA runtime
is linked statically). ``csrc/marshal.cc`` is compiled at the same time by the
host compiler, against the headers of the torch and Python that run this, where
they are there; its file has torch's version and a hash of its source in its name.
Nothing is installed anywhere else.

    python -m normalization_fwd_gb300.build [--force] [--verbose] [--ptxas-info]
"""

from __future__ import annotations

import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB_NAME = "libnormfuse.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
          "-I", os.path.join(ROOT, "include")]


def find_nvcc() -> str:
    cands = []
    for env in ("CUDA_HOME", "CUDA_PATH"):
        if os.environ.get(env):
            cands.append(os.path.join(os.environ[env], "bin", "nvcc"))
    cands.append("/usr/local/cuda/bin/nvcc")
    which = shutil.which("nvcc")
    if which:
        cands.append(which)
    for c in cands:
        if os.path.isfile(c) and os.access(c, os.X_OK):
            return c
    raise RuntimeError("nvcc not found: set CUDA_HOME or put nvcc on PATH")


def marshal_path() -> str:
    """Where the C++ part of the binding is, for this torch, this Python, its own
    source and the declarations that it calls: one of another state is not taken."""
    import torch
    state = hashlib.sha256()
    for path in (os.path.join(CSRC, "marshal.cc"), os.path.join(ROOT, "include", "normfuse.h")):
        if os.path.isfile(path):
            with open(path, "rb") as f:
                state.update(f.read() + b"\0")
    tag = f"{torch.__version__}-{sysconfig.get_config_var('SOABI')}-{state.hexdigest()[:8]}"
    return os.path.join(PKG, f"_marshal-{tag}.so")


def _marshal_commands():
    """(compile, link), or None where the C++ part cannot be built: it wants g++, a
    torch with CUDA and the headers of torch, Python and CUDA; the library does
    without it. Nothing of the library is linked in: the binding gives the
    addresses of the one that it has loaded."""
    import torch
    if torch.version.cuda is None or not shutil.which("g++"):
        return None
    at = os.path.dirname(torch.__file__)
    try:
        cuda = os.path.join(os.path.dirname(os.path.dirname(find_nvcc())), "include")
    except RuntimeError:
        return None
    dirs = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], cuda, os.path.join(ROOT, "include")]
    if not all(any(os.path.isfile(os.path.join(d, name)) for d in dirs)
               for name in ("c10/cuda/CUDAStream.h", "torch/csrc/autograd/python_variable.h", "Python.h",
                            "cuda_runtime_api.h")):
        return None
    obj = os.path.join(BUILD, "marshal.o")
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return (["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
             *[f"-I{d}" for d in dirs], "-c", os.path.join(CSRC, "marshal.cc"), "-o", obj],
            ["g++", "-shared", obj, "-o", marshal_path() + ".tmp", f"-L{os.path.join(at, 'lib')}", "-lc10",
             "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.cc")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    made = [LIB_PATH] + ([marshal_path()] if _marshal_commands() else [])
    if not all(os.path.isfile(p) for p in made):
        return False
    t = min(os.path.getmtime(p) for p in made)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False,
          jobs: int | None = None) -> str:
    """Compile and link the library; returns its path. Raises on failure."""
    if not force and not ptxas_info and up_to_date():
        return LIB_PATH
    nvcc = find_nvcc()
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *CFLAGS, *extra, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    jobs = jobs or min(len(_sources()), os.cpu_count() or 4)
    with ThreadPoolExecutor(max_workers=jobs + 1) as ex:
        commands = _marshal_commands()
        marshal = ex.submit(subprocess.run, commands[0], capture_output=True, text=True) if commands else None
        results = list(ex.map(compile_one, _sources()))
        marshal = marshal.result() if marshal else None
    failed = [(s, r) for s, _, r in results if r.returncode != 0]
    for s, _, r in results:
        if (verbose or ptxas_info) and (r.stdout or r.stderr):
            sys.stdout.write(r.stdout + r.stderr)
    if marshal is not None and marshal.returncode != 0:
        raise RuntimeError(f"g++ failed:\n--- marshal.cc\n{marshal.stdout}{marshal.stderr}")
    if failed:
        msg = "\n".join(f"--- {s}\n{r.stdout}{r.stderr}" for s, r in failed)
        raise RuntimeError(f"nvcc failed:\n{msg}")
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for _, o, _ in results]]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if commands:
        r = subprocess.run(commands[1], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
        os.replace(marshal_path() + ".tmp", marshal_path())
    elif verbose:
        print("the binding's C++ part is left out: no g++, no torch with CUDA, or no headers", flush=True)
    return LIB_PATH


if __name__ == "__main__":
    args = set(sys.argv[1:])
    path = build(force="--force" in args, verbose="--verbose" in args,
                 ptxas_info="--ptxas-info" in args)
    print(path)
