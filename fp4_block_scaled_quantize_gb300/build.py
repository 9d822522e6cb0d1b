"""Build libfp4gb300.so for sm_103a (GB300) with nvcc, in-tree.

Each CUDA translation unit is compiled in parallel into _build/, then linked
into fp4_block_scaled_quantize_gb300/_lib/libfp4gb300.so.  The quantizer
units are built with -fmad=false so no multiply-add is contracted into an FMA
(their arithmetic is specified as separately rounded binary32 operations).
csrc/bind.cpp, the serving calls' short way from Python into the library,
becomes _lib/_bind.so beside it (g++, the headers of the running interpreter
and its torch); it compiles while the CUDA units do.
"""
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libfp4gb300.so")
BIND = os.path.join(LIBDIR, "_bind.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC,
          "--expt-relaxed-constexpr"]
UNITS = {
    "abi.cu": [],
    "amax.cu": ["-fmad=false"],
    "quantize.cu": ["-fmad=false"],
    "remap.cu": ["-fmad=false"],
    "convert.cu": ["-fmad=false"],
    "dequant.cu": ["-fmad=false"],
    "gemm.cu": [],
    "gemm2.cu": [],
    "mmarate.cu": [],
    "matvec.cu": [],
    "append.cu": [],
    "attention.cu": [],
}


def nvcc():
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def cxx():
    return os.environ.get("CXX") or shutil.which("g++") or "c++"


def _torch():
    """The folder of the running interpreter's torch."""
    import torch
    return os.path.dirname(torch.__file__)


def _made_for():
    """What the binding's object depends on beside its sources."""
    import torch
    return f"{sys.implementation.cache_tag} torch {torch.__version__} {_torch()}"


def _read(path):
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def _stale(obj, deps):
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force=False, verbose=False, extra=()):
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    headers.append(os.path.join(INCLUDE, "fp4.h"))
    procs, host, objs, unbound = [], [], [], []
    for unit, flags in UNITS.items():
        src = os.path.join(CSRC, unit)
        obj = os.path.join(BUILD, unit.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc()] + ARCH + COMMON + flags + list(extra) + ["-c", src, "-o", obj]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            procs.append((unit, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                 stderr=subprocess.STDOUT, text=True)))
    bind, bind_obj, bind_for = (os.path.join(CSRC, "bind.cpp"), os.path.join(BUILD, "bind.o"),
                                os.path.join(BUILD, "bind.for"))
    try:
        made_for = _made_for()
        if force or _stale(bind_obj, [bind, os.path.join(INCLUDE, "fp4.h")]) or _read(bind_for) != made_for:
            host.append(("bind.cpp", subprocess.Popen(
                [cxx(), "-O2", "-Wall", "-std=c++17", "-fPIC", "-I" + INCLUDE,
                 "-I" + sysconfig.get_paths()["include"], "-isystem", os.path.join(_torch(), "include"),
                 "-isystem", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include"),
                 "-c", bind, "-o", bind_obj], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    except (ImportError, OSError) as e:  # no torch, no compiler
        unbound.append(f"bind.cpp ({e})")

    def wait(started):
        bad = []
        for unit, p in started:
            out, _ = p.communicate()
            if verbose or p.returncode:
                sys.stdout.write(out)
            if p.returncode:
                bad.append(unit)
        return bad

    failed = wait(procs)
    unbound += wait(host)
    if failed:
        raise RuntimeError("nvcc failed for " + ", ".join(failed))
    if force or procs or not os.path.exists(LIB) or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        subprocess.run([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs, check=True)
        os.replace(tmp, LIB)
    if unbound:  # the library, and all but the serving calls, do without it
        if os.path.exists(BIND):
            os.remove(BIND)  # made for another library
        raise RuntimeError("the library is built, but compilation failed for " + ", ".join(unbound))
    if force or _stale(BIND, [bind_obj, LIB]):
        tmp = BIND + ".tmp"
        subprocess.run([cxx(), "-shared", bind_obj, "-o", tmp, "-L" + LIBDIR, "-lfp4gb300",
                        "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(_torch(), "lib"), "-lc10",
                        "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"], check=True)
        os.replace(tmp, BIND)
        with open(bind_for, "w") as f:
            f.write(made_for)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
