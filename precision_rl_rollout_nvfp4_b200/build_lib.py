"""Build step of the CUDA library: compiles csrc/*.cu for sm_100a into
libnvfp4rac.so next to this file (in-tree, so it travels with the sources), and
csrc/host.cpp into the Python module _host.so."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SOURCES = ["api.cu", "quant.cu", "select.cu", "gemm.cu", "noalloc.cu",
           "api_mx4.cu", "mx4.cu", "mx4_gemm.cu", "mx4_pair.cu", "gated.cu"]
LIB = os.path.join(PKG, "libnvfp4rac.so")
# the index-checked build (NVFP4_CHECKS): same sources, every kernel store and
# gathered load tests its index
LIB_CHECKED = os.path.join(PKG, "libnvfp4rac_checked.so")
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-gencode", "arch=compute_100a,code=sm_100a",
         "-Xcompiler", "-fPIC", "-Xptxas", "-warn-spills"]


# the Python module that marshals the MXFP4 and gated calls (host.cpp; g++
# against torch's headers)
HOST = os.path.join(PKG, "_host.so")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def host_target() -> str:
    """What a host module has to be built against to serve this interpreter."""
    import torch
    return f"torch {torch.__version__} python {sys.version_info[0]}.{sys.version_info[1]}"


def host_needs_build(path: str = HOST) -> bool:
    """Missing, older than its sources, or built against another torch or Python
    (the module carries the name of what it was built against)."""
    if not os.path.exists(path):
        return True
    src = os.path.join(PKG, "csrc", "host.cpp")
    header = os.path.join(ROOT, "include", "nvfp4rac.h")
    if os.path.getmtime(path) <= max(os.path.getmtime(src), os.path.getmtime(header)):
        return True
    with open(path, "rb") as f:
        return host_target().encode() + b"\0" not in f.read()


def build_host(force: bool = False) -> str:
    if not force and not host_needs_build():
        return HOST
    src = os.path.join(PKG, "csrc", "host.cpp")
    import torch
    from torch.utils.cpp_extension import include_paths
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = [*include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include"),
           os.path.join(ROOT, "include")]
    # the system's g++, as nvcc takes it: a compiler that links its own libstdc++
    # statically gives the module a second one next to torch's
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DHOST_BUILT_AGAINST="{host_target()}"', *(f"-I{i}" for i in inc), src, "-o",
           HOST + ".tmp", f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-ltorch", "-ltorch_cuda", "-lc10", "-lc10_cuda",
           f"-Wl,-rpath,{lib}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stdout + res.stderr)
    os.replace(HOST + ".tmp", HOST)
    return HOST


def needs_build(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(PKG, "csrc", f) for f in os.listdir(os.path.join(PKG, "csrc"))]
    deps.append(os.path.join(ROOT, "include", "nvfp4rac.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _nvcc(args: list) -> str:
    res = subprocess.run([nvcc(), *args], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    return res.stdout + res.stderr


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    lib = LIB_CHECKED if checked else LIB
    build_host(force)
    if not force and not needs_build(lib):
        return lib
    # one object per source, compiled side by side, then one link
    flags = [*FLAGS, *(["-DNVFP4_CHECKS"] if checked else []), "-I", os.path.join(ROOT, "include")]
    with tempfile.TemporaryDirectory() as tmp:
        objs = [os.path.join(tmp, s + ".o") for s in SOURCES]
        with ThreadPoolExecutor(os.cpu_count() or 1) as pool:
            runs = list(pool.map(lambda a: _nvcc([*flags, "-c", os.path.join(PKG, "csrc", a[0]), "-o", a[1]]),
                                 zip(SOURCES, objs)))
        runs.append(_nvcc([*flags, "-shared", *objs, "-o", lib + ".tmp"]))
    out = "".join(runs)
    if verbose and out:
        print(out)
    os.replace(lib + ".tmp", lib)
    return lib


if __name__ == "__main__":
    print(build(force=True, verbose=True))
    print(build(force=True, verbose=True, checked=True))
