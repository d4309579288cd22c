"""Builds libmk.so (the C-ABI library) in-tree with nvcc for sm_103a.

Translation units compiled in parallel and linked into one shared library:
  csrc/mk_sched.cpp  host scheduler
  csrc/mk_api.cu     binding, launch and status (host)
  csrc/mk_kernel.cu  the persistent megakernel (batch-1 instances) and the RoPE table kernel (device)
  csrc/mk_kernel_batch.cu  the batch > 1 instance of the same kernel source (tensor-core matvec tiles)
  csrc/mk_linear.cu  the linear map with a fused epilogue (prompt path)
  csrc/mk_attend.cu  attention of query tokens over the KV cache (prompt path)
  csrc/mk_prefill.cu embedding, RMSNorm, RoPE and KV append of the prompt path
and beside it, with the host's C compiler, the Python module _mk_call, named for the interpreter it is built for:
  csrc/mk_python.c   argument handling of linear() and attend()
Where Python's headers are missing the module is left out, and that is done in Python.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from typing import List, Optional

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libmk.so")
CALL_SOURCE, CALL = os.path.join(CSRC, "mk_python.c"), os.path.join(HERE, "_mk_call" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
BUILD_DIR = os.path.join(HERE, "_build")
SOURCES = ["mk_sched.cpp", "mk_api.cu", "mk_kernel.cu", "mk_kernel_batch.cu", "mk_linear.cu", "mk_attend.cu",
           "mk_prefill.cu"]
HEADERS = ["mk_internal.h", "mk_ops.h", "mk_sm103.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _inputs() -> List[str]:
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "mk.h"), CALL_SOURCE, __file__]
    return files


def _python_headers() -> Optional[str]:
    path = sysconfig.get_paths()["include"]
    return path if os.path.exists(os.path.join(path, "Python.h")) else None


def up_to_date() -> bool:
    built = [LIB, CALL] if _python_headers() else [LIB]
    if not all(os.path.exists(f) for f in built):
        return False
    t = min(os.path.getmtime(f) for f in built)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link libmk.so unless it is newer than every source.  Returns its path."""
    if not force and not ptxas_info and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    common = ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", f"-I{INCLUDE}", f"-I{CSRC}"]

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, src + ".o")
        cmd = [nvcc, *common, *ARCH, "-lineinfo", "-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cpp"):
            cmd = [nvcc, *common, "-x", "c++", "-c", os.path.join(CSRC, src), "-o", obj]
        if ptxas_info and src in ("mk_kernel.cu", "mk_linear.cu", "mk_attend.cu"):
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    def compile_call() -> None:
        old = os.path.join(HERE, "_mk_call.so")   # (a module without a tag would load in any interpreter)
        if old != CALL and os.path.exists(old):
            os.remove(old)
        headers = _python_headers()
        if not headers:
            sys.stderr.write("Python.h not found: linear() and attend() take their arguments in Python\n")
            return
        tmp = CALL + f".{os.getpid()}.tmp"
        r = subprocess.run([os.environ.get("CC", "gcc"), "-O2", "-Wall", "-shared", "-fPIC", f"-I{headers}",
                            f"-I{INCLUDE}", CALL_SOURCE, "-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"C compiler failed on mk_python.c:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, CALL)

    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        call = ex.submit(compile_call)
        objs = list(ex.map(compile_one, SOURCES))
        call.result()
    tmp = LIB + f".{os.getpid()}.tmp"
    link = [nvcc, *ARCH, "-shared", "-cudart", "shared", *objs, "-o", tmp]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True, ptxas_info="--ptxas" in sys.argv))
