"""Build libwq.so (the CUDA library behind include/wq.h) in-tree for sm_100a.

Each .cu under csrc/ is compiled to an object in _build/ with nvcc
(-gencode arch=compute_100a,code=sm_100a, -O3, -lineinfo, no fast-math: the
quantisers rely on IEEE division and round-to-nearest-even), then linked
into group_wise_weight_b200/libwq.so.  The binding of the prompt-side calls
(csrc/wq_torch.cpp, a CPython extension on torch's headers) is compiled with
g++ into group_wise_weight_b200/_wq_torch.so and linked against libwq.so
beside it.  Objects are rebuilt only when a source or header is newer; the
binding also when the torch or Python that it was compiled against differs
from the present one (recorded in _build/ beside the objects).  Where g++ or
the headers of Python or torch are missing the binding is left out with a
warning: libwq.so and every call that goes through it alone need none of
them, and the prompt-side calls raise.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libwq.so")
BINDING = os.path.join(PKG, "_wq_torch.so")
BINDING_STAMP = os.path.join(BUILD, "wq_torch.stamp")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libwq")
    return path


def _deps():
    return (glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")))


def _stale(target: str, inputs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in inputs)


def _binding_stamp() -> str:
    """What a compiled binding is bound to: torch's C++ classes, Python's ABI, and how it was compiled (no paths of this
    checkout, which may move)."""
    import torch

    return "\n".join([f"torch {torch.__version__} {torch.version.git_version} cuda {torch.version.cuda}",
                      f"cxx11abi {int(torch.compiled_with_cxx11_abi())}",
                      f"python {sys.version} {sysconfig.get_config_var('SOABI')}"]
                     + [a for a in _binding_command("") if not os.path.isabs(a.removeprefix("-I").removeprefix("-L"))])


def _read(path: str):
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def _torch_home() -> str:
    import torch

    return os.path.dirname(torch.__file__)


def _binding_lacks():
    """What the binding cannot be compiled without and this machine does not have."""
    headers = [os.path.join(sysconfig.get_paths()["include"], "Python.h"),
               os.path.join(_torch_home(), "include", "torch", "csrc", "autograd", "python_variable.h")]
    return [h for h in headers if not os.path.exists(h)] + ([] if shutil.which("g++") else ["g++"])


def _binding_command(src: str):
    import torch

    home = _torch_home()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    libs = os.path.join(home, "lib")
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
            + [f"-I{d}" for d in inc] + [src, "-o", BINDING + ".tmp", f"-L{PKG}", "-l:libwq.so", "-Wl,-rpath,$ORIGIN",
                                         f"-L{libs}", "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"])


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = _deps()
    objs, jobs = [], []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + deps):
            cmd = [nvcc()] + ARCH + NVCC_FLAGS + (["-Xptxas", "-v"] if ptxas_info else []) + ["-c", src, "-o", obj]
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        return r.stdout + r.stderr

    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
            for out in ex.map(run, jobs):
                if verbose and out.strip():
                    print(out)
    if force or jobs or _stale(LIB, objs):
        cmd = [nvcc()] + ARCH + ["-shared", "-o", LIB + ".tmp"] + objs + ["-lcudart"]
        run(cmd)
        os.replace(LIB + ".tmp", LIB)
    binding_src = os.path.join(CSRC, "wq_torch.cpp")
    stamp = _binding_stamp()
    if (force or _stale(BINDING, [binding_src] + glob.glob(os.path.join(ROOT, "include", "*.h")))
            or _read(BINDING_STAMP) != stamp):
        lacks = _binding_lacks()
        if lacks:
            if os.path.exists(BINDING):  # it belongs to other sources or another torch or Python
                os.remove(BINDING)
            warnings.warn(f"{os.path.basename(BINDING)}, the binding of the prompt-side calls, is left out: "
                          f"{', '.join(lacks)} not found")
            return LIB
        run(_binding_command(binding_src))
        os.replace(BINDING + ".tmp", BINDING)
        with open(BINDING_STAMP, "w") as f:
            f.write(stamp)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
