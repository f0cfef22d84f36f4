"""Build libdaa.so in-tree with nvcc for sm_103a (no cmake), and the module that
hands torch tensors to some of its calls (``csrc/binding.cpp``, with g++).

Each CUDA translation unit compiles in parallel to an object file under
``_build/``; they link into one shared library with the CUDA runtime linked
statically.  The module links against it and against the torch that is installed,
and is built again for another one.  Rebuilds only what changed.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libdaa.so")
BINDING = os.path.join(BUILD, "_binding.so")
SOURCES = ["api.cu", "append.cu", "decode.cu", "merge.cu", "prefill.cu", "prefill_pair.cu", "noalloc.cu",
           "api_q4.cu", "append_q4.cu", "decode_q4.cu", "step_table.cu",
           "api_rope.cu", "rope.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    hs.append(os.path.join(ROOT, "include", "daa.h"))
    return hs


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd, verbose):
    tool = os.path.basename(cmd[0])
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"{tool} could not be run: {e}") from e
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        last = (r.stderr.strip().splitlines() or [""])[-1]
        raise RuntimeError(f"{tool} failed: {' '.join(cmd[-3:])}: {last}")


def build(verbose: bool = False, force: bool = False) -> str:
    """The library's path.  Without torch, its headers or Python's, only the module is
    missing: the library is built all the same, and the calls that need the module
    raise an ImportError with the reason."""
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    headers = _headers()
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([nvcc, *ARCH, *FLAGS, "-c", s, "-o", o])

    with ThreadPoolExecutor(max_workers=min(len(jobs) + 1, os.cpu_count() or 4)) as ex:
        module = ex.submit(_compile_module, verbose, force)  # beside nvcc's work
        list(ex.map(lambda cmd: _run(cmd, verbose), jobs))
        if force or jobs or _stale(LIB, objs):
            tmp = LIB + f".tmp{os.getpid()}"
            _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], verbose)
            os.replace(tmp, LIB)
    error = os.path.join(BUILD, "_binding.error")  # why there is no module, read by the package
    try:
        _link_module(*module.result(), verbose, force)
    except (ImportError, RuntimeError) as e:
        sys.stderr.write(f"_binding.so is not built, and calls that need it will fail: {e}\n")
        _remove(BINDING)  # of another library or torch
        with open(error, "w") as f:
            f.write(str(e))
    else:
        _remove(error)
    return LIB


def _remove(path):
    if os.path.exists(path):
        os.remove(path)


def _compile_module(verbose, force):
    """(torch, tag, object file): the object file goes by the torch and Python that it is for."""
    import torch
    tag = f"{torch.__version__}-{sys.version_info[0]}.{sys.version_info[1]}".replace("/", "_")
    src, obj = os.path.join(CSRC, "binding.cpp"), os.path.join(BUILD, f"binding-{tag}.o")
    if force or _stale(obj, [src, os.path.join(ROOT, "include", "daa.h")]):
        _run([_gxx(), *_torch_flags(torch), "-c", src, "-o", obj], verbose)
    return torch, tag, obj


def _link_module(torch, tag, obj, verbose, force):
    stamp = os.path.join(BUILD, f"binding-{tag}.linked.o")  # empty: which torch the module is linked for
    if not force and not _stale(BINDING, [obj, LIB]) and os.path.exists(stamp):
        return
    tmp = BINDING + f".tmp{os.getpid()}"
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    _run([_gxx(), "-shared", "-o", tmp, obj, f"-L{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
          f"-L{BUILD}", "-l:libdaa.so", "-Wl,-rpath,$ORIGIN"], verbose)
    for f in os.listdir(BUILD):
        if f.endswith(".linked.o"):
            os.remove(os.path.join(BUILD, f))
    os.replace(tmp, BINDING)
    open(stamp, "w").close()


def _gxx():
    return shutil.which("g++") or "g++"


def _torch_flags(torch):
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    return ["-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-I{d}" for d in (inc, os.path.join(inc, "torch", "csrc", "api", "include"),
                                 sysconfig.get_path("include"), os.path.join(cuda, "include")))]


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
