"""Build the in-tree CUDA library ``_build/libnvfp4w4a16.so`` for sm_103a, and the
Python module ``_build/_nvfp4_binding.so`` over it.

Each ``csrc/*.cu`` is compiled by nvcc in parallel and the objects are linked
into one shared library (static CUDA runtime, no relocatable device code);
``csrc/binding.cpp`` is compiled beside them by g++ against torch's headers.
Each of the two is rebuilt only when a source or header of its own is newer, the
module also for another torch or Python than it was built for.  The library needs
nvcc alone: where the module cannot be built, build() warns and leaves the library.

    python -m w4a16_nvfp4_weight_gb300.build_lib [--force]
"""

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


def _newer(target, deps):
    """Whether `target` is there and no older than any of `deps`."""
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps + [os.path.abspath(__file__)])


def _headers():
    return glob.glob(os.path.join(ROOT, "include", "*.h"))


def library_up_to_date():
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + _headers())


def _binding_abi():
    """What the module's C++ and Python interfaces go by."""
    import torch
    return f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')}"


def binding_abi_built():
    """_binding_abi() of the torch and Python that the module in place was built for, or None."""
    try:
        with open(BINDING + ".abi") as f:
            return f.read().strip()
    except OSError:
        return None


def binding_up_to_date():
    return _newer(BINDING, [BINDING_SRC] + _headers()) and binding_abi_built() == _binding_abi()


def up_to_date():
    return library_up_to_date() and binding_up_to_date()


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
    with open(BINDING + ".abi", "w") as f:
        f.write(_binding_abi() + "\n")


def _link_library(objs):
    tmp = LIB + ".tmp"
    r = subprocess.run([_nvcc()] + ARCH + ["-shared", "-o", tmp] + objs, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force=False, verbose=False):
    """Compile and link the library and its Python module, each where it is out of date;
    returns the library's path.  A library that cannot be built raises; a module that
    cannot be is a warning (the operators of layer_ops then raise when called)."""
    library, binding = force or not library_up_to_date(), force or not binding_up_to_date()
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources() if library else []
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        module = ex.submit(_compile_binding) if binding else None
        results = list(ex.map(lambda s: _compile(s, verbose), srcs))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    if library:
        _link_library([o for o, _ in results])
    if binding:
        try:
            _link_binding(module.result())
        except (RuntimeError, OSError) as e:
            if os.path.exists(BINDING):                # one of older sources must not stand in
                os.remove(BINDING)
            warnings.warn(f"the library is built, its Python module is not: {e}")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
