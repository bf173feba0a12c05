"""Build libdkv.so in-tree (nvcc for sm_103a, one object per .cu in parallel) and
the Python binding beside it (g++, against the installed torch).

    python -m decode_attention_paged_kv_gb300.build [--force]
"""

from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libdkv.so")
BINDING = os.path.join(BUILD, "_binding.so")
BINDING_STAMP = os.path.join(BUILD, "_binding.for")  # the torch and Python it was made for
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CXX = os.environ.get("CXX", "g++")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I" + INCLUDE,
         "--expt-relaxed-constexpr"]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _newer(paths, than: str) -> bool:
    t = os.path.getmtime(than)
    return any(os.path.getmtime(p) > t for p in paths)


def _headers():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
        os.path.join(INCLUDE, "dkv.h")]


def _library_stale() -> bool:
    return not os.path.exists(LIB) or _newer(sources() + _headers(), LIB)


def _made_for() -> str:
    """What the binding's compilation depends on besides its source."""
    import torch
    return f"torch {torch.__version__} at {os.path.dirname(torch.__file__)}, python {sys.version}\n"


def _binding_stale() -> bool:
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_STAMP):
        return True
    if _newer([BINDING_SOURCE, os.path.join(INCLUDE, "dkv.h")], BINDING):
        return True
    with open(BINDING_STAMP) as f:
        return f.read() != _made_for()


def needs_build() -> bool:
    return _library_stale() or _binding_stale()


def build(force: bool = False, verbose: bool = False) -> str:
    """The path of libdkv.so, after building what is older than its sources (the
    binding: or was made for another torch or Python)."""
    library, binding = force or _library_stale(), force or _binding_stale()
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        _run([NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj], f"nvcc for {src}", verbose)
        return obj

    with ThreadPoolExecutor(max_workers=min(9, os.cpu_count() or 4)) as ex:
        made = ex.submit(_compile_binding, verbose) if binding else None
        if library:  # (whatever becomes of the binding, which users of the C ABI do not need)
            objs = list(ex.map(compile_one, sources()))
            tmp = LIB + f".tmp{os.getpid()}"
            _run([NVCC, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
                  "-Xlinker", "-rpath=/usr/local/cuda/lib64"], "the link", verbose)
            os.replace(tmp, LIB)
        if made is not None:
            _link_binding(made.result(), verbose)
    return LIB


def _run(cmd, what: str, verbose: bool = False) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_binding(verbose: bool) -> str:
    import torch
    torch_include = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda_include = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    obj = os.path.join(BUILD, "binding.o")
    _run([CXX, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-I" + INCLUDE, "-I" + torch_include,
          "-I" + os.path.join(torch_include, "torch", "csrc", "api", "include"),
          "-I" + sysconfig.get_paths()["include"], "-I" + cuda_include,
          "-c", BINDING_SOURCE, "-o", obj], "the binding's compilation", verbose)
    return obj


def _link_binding(obj: str, verbose: bool) -> None:
    import torch
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    _run([CXX, "-shared", obj, "-o", tmp, "-L" + BUILD, "-l:libdkv.so", "-Wl,-rpath,$ORIGIN",
          "-L" + torch_lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
          "-Wl,-rpath," + torch_lib], "the binding's link", verbose)
    os.replace(tmp, BINDING)
    with open(BINDING_STAMP, "w") as f:
        f.write(_made_for())


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
