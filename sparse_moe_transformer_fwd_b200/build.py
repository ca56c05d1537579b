"""Build the CUDA library libmoe_fwd.so in-tree for sm_100a with nvcc, and, where
this Python's headers are, the binding's C module (csrc/binding.c) beside it.

The library is the product: every step of the layer runs in its kernels.
cudart is linked statically and the driver entry point for tensor-map
encoding is fetched at run time, so the library loads on a machine without
a GPU driver (its calls then fail with MOE_ERR_CUDA)."""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe_fwd.so")
SOURCES = ["api.cu", "router.cu", "permute.cu", "quant.cu", "combine.cu", "gemm_sm100.cu",
           "route_noalloc.cu", "ep.cu", "linear.cu", "few.cu"]
BINDING = os.path.join(HERE, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
INCLUDE = sysconfig.get_paths()["include"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def _deps_mtime() -> float:
    root = os.path.dirname(HERE)
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(root, "include", "moe_fwd.h")]
    return max(os.path.getmtime(f) for f in files)


def build(force: bool = False, verbose: bool = False) -> str:
    with_binding = os.path.exists(os.path.join(INCLUDE, "Python.h"))
    made = (LIB, BINDING) if with_binding else (LIB,)
    if not force and all(os.path.exists(f) and os.path.getmtime(f) >= _deps_mtime() for f in made):
        return LIB
    os.makedirs(OUT, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(OUT, src.replace(".cu", ".o"))
        cmd = [NVCC, *FLAGS, "-Xptxas", "-v", "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xcompiler", "-fPIC",
           *[o for o, _ in results], "-o", tmp]
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    if not with_binding:  # the package does without; an old one may be of other structures
        if os.path.exists(BINDING):
            os.remove(BINDING)
        return LIB
    tmp = BINDING + ".tmp%d" % os.getpid()
    subprocess.check_call(["gcc", "-O2", "-Wall", "-shared", "-fPIC", "-I" + INCLUDE, os.path.join(CSRC, "binding.c"), "-o", tmp])
    os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))
