"""Build the in-tree CUDA library ``_build/libnvfp4w4a16.so`` for sm_103a, and the
Python module ``_build/_nvfp4_binding.so`` over it.

Each ``csrc/*.cu`` is compiled by nvcc in parallel and the objects are linked
into one shared library (static CUDA runtime, no relocatable device code);
``csrc/binding.cpp`` is compiled beside them by g++ against torch's headers.
Rebuilds only when a source or header is newer than the libraries.

    python -m w4a16_nvfp4_weight_gb300.build_lib [--force]
"""

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libnvfp4w4a16.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(BUILD, "_nvfp4_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "-I", os.path.join(ROOT, "include")]


def _nvcc():
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return exe


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + [BINDING_SRC] + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]


def up_to_date():
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(d) <= t for d in _deps())


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [_nvcc()] + ARCH + FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch_dir():
    import torch
    return os.path.dirname(os.path.abspath(torch.__file__))


def _compile_binding():
    torch_dir = _torch_dir()
    inc = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           os.path.join(ROOT, "include")]
    obj = os.path.join(BUILD, "binding.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden"] + [x for d in inc for x in ("-isystem", d)] +
         ["-c", BINDING_SRC, "-o", obj], "g++ binding.cpp")
    return obj


def _link_binding(obj):
    lib = os.path.join(_torch_dir(), "lib")
    _run(["g++", "-shared", "-o", BINDING + ".tmp", obj, "-L" + BUILD, "-L" + lib, "-lnvfp4w4a16", "-ltorch_python",
          "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib], "linking the binding")
    os.replace(BINDING + ".tmp", BINDING)


def build(force=False, verbose=False):
    """Compile and link the library and its Python module; returns the library's path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(lambda s: _compile(s, verbose), srcs))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp"
    cmd = [_nvcc()] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
