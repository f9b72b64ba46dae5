"""Build the SCAPE CUDA library (libscape.so) in-tree for sm_103a, and the torch
binding of its training-layer operators (_layers_torch.so).

Each translation unit under csrc/ is compiled in parallel (.cu by nvcc, the
binding by g++), then linked into sparse_communication_sharded_gb300/_build/.
No CMake; one -gencode (compute_103a -> sm_103a).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libscape.so")
BINDING_SRC = os.path.join(CSRC, "layers_torch.cpp")
BINDING = os.path.join(BUILD, "_layers_torch.so")
BINDING_FOR = os.path.join(BUILD, "_layers_torch.for")  # what the binding was built against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc():
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + [BINDING_SRC] + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def is_stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return any(os.path.getmtime(p) > t for p in _deps()) or binding_mismatch() is not None


def _here() -> str:
    """The interpreter and torch that a binding built now would fit."""
    import torch
    return (f"python {sys.version_info.major}.{sys.version_info.minor}, torch {torch.__version__}, "
            f"C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}")


def binding_mismatch() -> str | None:
    """Why the built binding does not fit this process, or None: it uses torch's C++
    classes, whose layout another torch may have changed without a missing symbol."""
    try:
        with open(BINDING_FOR) as f:
            built = f.read()
    except OSError:
        built = "unknown"
    return None if built == _here() else f"built for {built}; this is {_here()}"


def _torch_dir():
    import torch
    return os.path.dirname(torch.__file__), int(torch._C._GLIBCXX_USE_CXX11_ABI)


def _compile_binding():
    torch_dir, abi = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda"
    obj = os.path.join(BUILD, "layers_torch.o")
    inc = [INCLUDE, os.path.join(torch_dir, "include"),
           os.path.join(torch_dir, "include/torch/csrc/api/include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
           *[f"-I{d}" for d in inc], "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stderr}")
    return obj


def _link_binding(obj):
    lib = os.path.join(_torch_dir()[0], "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, f"-L{BUILD}", "-lscape", f"-L{lib}", "-ltorch_python",
           "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN",
           f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    if os.path.exists(BINDING_FOR):
        os.remove(BINDING_FOR)  # no moment at which it stands for another binding
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(_here())


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and not is_stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(compile_one, _sources()))
        binding_obj = binding.result()
    if verbose_ptxas:
        for _, log in results:
            sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding_obj)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
