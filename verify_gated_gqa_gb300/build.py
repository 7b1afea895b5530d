"""Build libga_attn.so in-tree: one nvcc per translation unit (in parallel) for sm_103a,
then one shared-library link, and beside it the native half of the torch binding
(_native.so, plain C++ against torch's headers). No CMake; a rebuild only recompiles
changed units. The library needs nvcc alone: it is linked whatever becomes of the module, which is
left out where there is no torch."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libga_attn.so")
NATIVE_SRC = os.path.join(CSRC, "ga_native.cpp")
NATIVE = os.path.join(PKG, "_native.so")
SOURCES = ["ga_host.cu", "ga_prologue.cu", "ga_attn.cu", "ga_mask.cu", "ga_quant.cu",
           "ga_select.cu", "ga_kv4.cu", "ga_plan.cu", "ga_verify4.cu", "ga_decode4.cu",
           "ga_pages.cu", "ga_kv8.cu", "ga_verify8.cu", "ga_verify8_rows.cu",
           "ga_debug.cu"]
HEADERS = ["ga_internal.h", "ga_numerics.cuh", "ga_q4.cuh", "ga_q8.cuh", "ga_sm100.cuh", "ga_v4.cuh", "ga_v8.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _newest_dep() -> float:
    deps = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "ga_attn.h")]
    return max(os.path.getmtime(p) for p in deps)


def _native_commands(obj: str):
    """Compile and link commands of the native binding against the installed torch, and a text that
    changes with everything they depend on beside the sources."""
    import torch

    tdir = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [os.path.join(tdir, "include"), os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", *[f"-I{d}" for d in inc],
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
                "-c", NATIVE_SRC, "-o", obj]
    link = ["g++", "-shared", "-o", NATIVE, obj, "-L", PKG, "-l:libga_attn.so",
            "-L", os.path.join(tdir, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
            "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    key = "\n".join([torch.__version__, str(sysconfig.get_config_var("SOABI")), " ".join(compile_),
                     " ".join(link)])
    return compile_, link, key


def _read(path: str) -> str:
    if not os.path.exists(path):
        return ""
    with open(path) as f:
        return f.read()


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    dep_time = _newest_dep()
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        stale = force or not os.path.exists(o) or os.path.getmtime(o) < max(os.path.getmtime(s), dep_time)
        if stale:
            jobs.append([nvcc, *ARCH, *FLAGS, "-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed for {cmd[-3]}")

    native_obj = os.path.join(BUILD, "ga_native.o")
    # the module holds torch's and Python's types: the stamp names the ones it was compiled against
    native_stamp = os.path.join(BUILD, "ga_native.stamp")
    native_dep = max(os.path.getmtime(NATIVE_SRC),
                     os.path.getmtime(os.path.join(ROOT, "include", "ga_attn.h")))
    try:
        native_compile, native_link, native_key = _native_commands(native_obj)
        native = (force or not os.path.exists(NATIVE) or not os.path.exists(native_obj) or
                  min(os.path.getmtime(NATIVE), os.path.getmtime(native_obj)) < native_dep or
                  _read(native_stamp) != native_key)
    except ImportError:
        native = False
        sys.stderr.write("torch is not installed: _native.so is not built\n")

    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 1))) as ex:
        native_job = ex.submit(run, native_compile) if native else None
        list(ex.map(run, jobs))
        if jobs or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
            run([nvcc, *ARCH, "-shared", "-o", LIB, *objs, "-lcudart"])
        if native:
            native_job.result()
            run(native_link)
            with open(native_stamp, "w") as f:
                f.write(native_key)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
