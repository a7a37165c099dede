"""Build libgdn.so (the C-ABI library of sm_103a CUDA kernels) in-tree, and
``_gdn_torch``, the host-side Python entry of the layer operators.

Each translation unit under csrc/ is compiled by its own process (in parallel),
then linked into ``_build/libgdn.so`` (the .cu files; only sm_103a is targeted)
and ``_build/_gdn_torch.so`` (gdn_torch.cpp, against the installed torch's
headers; it is rebuilt when torch or Python changes). The library needs neither
torch nor that module: without torch only the library is built, and it is linked
before the module.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libgdn.so")
INCLUDE = os.path.join(ROOT, "include")
EXT = os.path.join(OUT, "_gdn_torch.so")
EXT_SRC = os.path.join(CSRC, "gdn_torch.cpp")
EXT_FOR = os.path.join(OUT, "_gdn_torch.for")  # what the extension was built against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE,
         "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdn.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _torch_root():
    """Where torch is installed, or None."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def _built_for() -> str:
    with open(os.path.join(_torch_root(), "version.py")) as f:
        return sys.version + "\n" + f.read()


def _older(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _stale() -> bool:
    return _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def _ext_stale() -> bool:
    return _older(EXT, [EXT_SRC] + glob.glob(os.path.join(INCLUDE, "*.h"))) or not ext_fits()


def ext_fits() -> bool:
    """Whether _gdn_torch was built against this Python and torch."""
    if not os.path.exists(EXT_FOR):
        return False
    with open(EXT_FOR) as f:
        return f.read() == _built_for()


def _ext_compile(obj: str) -> list:
    torch = os.path.join(_torch_root(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE]
    for d in (torch, os.path.join(torch, "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"], cuda):
        cmd += ["-isystem", d]
    return cmd + ["-c", EXT_SRC, "-o", obj]


def _ext_link(obj: str, to: str) -> list:
    lib = os.path.join(_torch_root(), "lib")
    return ["g++", "-shared", "-o", to, obj, "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
            "-lc10_cuda", LIB, "-Wl,-rpath,$ORIGIN"]


def build(force: bool = False, verbose: bool = False) -> str:
    kernels = force or _stale()
    ext = _torch_root() is not None and (force or _ext_stale())
    if not kernels and not ext:
        return LIB
    os.makedirs(OUT, exist_ok=True)
    cc = nvcc()
    procs = []
    objs = []
    for src in sources() if kernels else []:
        obj = os.path.join(OUT, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [cc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                            stderr=subprocess.STDOUT, text=True)))
    ext_obj = os.path.join(OUT, "gdn_torch.o")
    if ext:
        procs.append((EXT_SRC, subprocess.Popen(_ext_compile(ext_obj), stdout=subprocess.PIPE,
                                                stderr=subprocess.STDOUT, text=True)))
    failed = set()
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode:
            sys.stdout.write(out)
        if p.returncode:
            failed.add(src)
    if kernels and failed <= {EXT_SRC}:
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.check_call([cc, *ARCH, "-shared", "-Xlinker", "-soname=libgdn.so", "-o", tmp,
                               *objs])
        os.replace(tmp, LIB)
    if failed:
        raise RuntimeError("compilation failed for: " + ", ".join(sorted(failed)))
    if ext:
        tmp = EXT + f".tmp{os.getpid()}"
        subprocess.check_call(_ext_link(ext_obj, tmp))
        os.replace(tmp, EXT)
        with open(EXT_FOR, "w") as f:
            f.write(_built_for())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
