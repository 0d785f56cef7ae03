"""Build step for the CUDA library: compiles csrc/*.cu for sm_100a with nvcc and links
libgdn_b200.so next to this file (in-tree, so it travels with the repository), and csrc/host.cpp, the
Python calls' host path, into _gdn_host.so."""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
OUT = os.path.join(HERE, "libgdn_b200.so")
OBJ = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found")
    return p


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


HOST_SRC = os.path.join(CSRC, "host.cpp")
HOST_OUT = os.path.join(HERE, "_gdn_host.so")


def build_host() -> str | None:
    """Compiles csrc/host.cpp (the calls' path from Python tensors to the C entry points) against this interpreter
    and its torch. Returns None, with the compiler's words on stderr, where it cannot be: the binding
    then makes its calls through ctypes alone."""
    deps = max(os.path.getmtime(f) for f in (HOST_SRC, os.path.join(ROOT, "include", "gdn.h"), __file__))
    if os.path.exists(HOST_OUT) and os.path.getmtime(HOST_OUT) >= deps:
        return HOST_OUT
    spec = importlib.util.find_spec("torch")
    torch_dir = list(spec.submodule_search_locations)[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = HOST_OUT + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-I" + os.path.join(torch_dir, "include"), "-I" + os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-I" + os.path.join(cuda, "include"), "-I" + sysconfig.get_paths()["include"], HOST_SRC, "-o", tmp,
           "-L" + os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        print("host path not built: %s" % e, file=sys.stderr)
        return None
    if r.returncode != 0:
        print("host path not built:\n" + r.stderr[-4000:], file=sys.stderr)
        return None
    os.replace(tmp, HOST_OUT)
    return HOST_OUT


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "host.cpp"] + [os.path.join(ROOT, "include", "gdn.h"),
                                                                  __file__]
    return max(os.path.getmtime(f) for f in files)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    out = build_library(force, verbose, extra)
    build_host()
    return out


def build_library(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and os.path.exists(OUT) and os.path.getmtime(OUT) >= _deps_mtime():
        return OUT
    os.makedirs(OBJ, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(OBJ, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = OUT + ".tmp%d" % os.getpid()
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))
