"""Build libmoe_gb300.so in-tree for sm_103a (nvcc, one -gencode, parallel TUs), and
_binding.so, the Python entries of the decoder-block operators (g++, against torch).
The library needs nvcc only: it is linked first, and where the binding's own needs
(g++, Python.h, torch with its headers) are missing, it is left out with a warning."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe_gb300.so")
BINDING = os.path.join(HERE, "_binding.so")
SOURCES = ["moe_api.cu", "moe_route.cu", "moe_gemm.cu", "moe_gemm_decode.cu", "moe_gemm_mx.cu", "moe_gate.cu", "moe_append.cu",
           "moe_attend.cu", "moe_pages.cu", "moe_tree.cu", "moe_tree_bf16.cu",
           "moe_tree_fp16.cu", "moe_tree_e4m3.cu"]
HEADERS = ["moe_device.cuh", "moe_attend.cuh", "moe_tree.cuh", "moe_internal.h", "moe_scan.cuh"]
NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xptxas", "-v"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale() -> bool:
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(ROOT, "include", "moe_gb300.h")]
    return not os.path.exists(LIB) or any(os.path.getmtime(d) > os.path.getmtime(LIB) for d in deps)


def _binding_missing() -> str:
    """What the binding cannot be built without and is not here, or ''."""
    if not shutil.which("g++"):
        return "g++"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    try:
        import torch
    except ImportError:
        return "torch"
    if not os.path.exists(os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc", "Exceptions.h")):
        return "torch's headers"
    return ""


def _binding_made_for() -> str:
    import torch
    return f"torch {torch.__version__} python {sys.version.split()[0]}"


def _stamp() -> str:
    return os.path.join(BUILD, "binding.for")


def binding_current() -> bool:
    """Whether _binding.so is there and was made for this torch and Python (their C++ interfaces
    change between versions)."""
    return os.path.exists(BINDING) and os.path.exists(_stamp()) and open(_stamp()).read() == _binding_made_for()


def _binding_stale() -> bool:
    deps = [os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "moe_gb300.h")]
    return not binding_current() or any(os.path.getmtime(d) > os.path.getmtime(BINDING) for d in deps)


GEMM_LAUNCH_REGS = 168  # must match GemmCfg<...>::LAUNCH_REGS (setmaxnreg budget)


def _check_gemm_registers(log_path: str) -> None:
    """The prefill GEMMs move registers between warpgroups with setmaxnreg; the
    split balances only if each kernel launches with exactly 168 registers."""
    import re
    text = open(log_path).read()
    found = re.findall(r"Compiling entry function '(_ZN3moe15moe_gemm_kernelILb[01]E[^']*)'.*?Used (\d+) registers", text,
                       re.S)
    if len(found) != 2 or any(int(n) != GEMM_LAUNCH_REGS for _, n in found):
        raise RuntimeError(f"prefill GEMMs compiled to {[n for _, n in found]} registers, expected {GEMM_LAUNCH_REGS}")
    if "setmaxnreg" in text and "ignored" in text:
        raise RuntimeError("ptxas ignored setmaxnreg in a prefill GEMM")


def _compile_binding() -> str:
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD, "binding.o")
    cuda = os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda"
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj, "-I" + inc,
                        "-I" + os.path.join(inc, "torch", "csrc", "api", "include"),
                        "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"),
                        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stderr[-4000:]}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, "-L" + HERE, "-l:libmoe_gb300.so", "-Wl,-rpath,$ORIGIN", "-L" + lib,
                        "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"], capture_output=True,
                       text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, BINDING)
    with open(_stamp(), "w") as f:
        f.write(_binding_made_for())


def build(force: bool = False, verbose: bool = False) -> str:
    missing = _binding_missing()
    library = force or _stale()
    binding = not missing and (force or _binding_stale())
    if missing:
        warnings.warn(f"no {missing}: the decoder-block operators (route_experts, rotate_append, paged_attention and those "
                      "beside them) get no Python entries (the C library is not affected)", stacklevel=2)
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        with open(os.path.join(BUILD, src + ".log"), "w") as f:
            f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr[-4000:]}")
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding_obj = ex.submit(_compile_binding) if binding else None
        if library:
            objs = list(ex.map(compile_one, SOURCES))
            _check_gemm_registers(os.path.join(BUILD, "moe_gemm.cu.log"))
            tmp = LIB + ".tmp"
            r = subprocess.run([nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-o", tmp, *objs],
                               capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
            os.replace(tmp, LIB)
        if binding:
            _link_binding(binding_obj.result())
    if verbose and library:
        for src in SOURCES:
            print(open(os.path.join(BUILD, src + ".log")).read())
    return LIB


if __name__ == "__main__":
    build(force=True, verbose=True)
