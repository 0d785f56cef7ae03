"""Build step for the CUDA library: compiles csrc/*.cu for sm_100a with nvcc and links
libgdn_b200.so next to this file (in-tree, so it travels with the repository), and csrc/host.cpp, the
Python calls' host path, into _gdn_host.<this Python's ABI>.so where it can be."""
from __future__ import annotations

import hashlib
import importlib.util
import os
import re
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
HOST_OUT = os.path.join(HERE, "_gdn_host" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))   # (named for this Python's ABI)
HOST_KEY = os.path.join(OBJ, "_gdn_host.key")   # what it was built from


def host_key(torch_version: str) -> str:
    """What a built host path holds good for: its sources, this interpreter and its torch (whose tensor accessors it
    inlines). It is compiled in, and the binding uses no other."""
    h = hashlib.sha256()
    for f in (HOST_SRC, os.path.join(ROOT, "include", "gdn.h"), __file__):
        with open(f, "rb") as src:
            h.update(src.read())
    return "%s torch-%s %s" % (sys.implementation.cache_tag, torch_version, h.hexdigest()[:24])


def _torch_version(torch_dir: str) -> str:
    with open(os.path.join(torch_dir, "version.py")) as f:   # (importing torch takes seconds)
        return re.search(r"__version__\s*=\s*['\"]([^'\"]+)", f.read()).group(1)


def build_host(force: bool = False) -> str | None:
    """Compiles csrc/host.cpp (the calls' path from Python tensors to the C entry points) against this interpreter
    and its torch. Returns None, with the reason on stderr and no file left in place, where it cannot be: the binding
    then makes its calls through ctypes alone."""
    untagged = os.path.join(os.path.dirname(HOST_OUT), "_gdn_host.so")   # a module of any Python, which import would take too

    def not_built(why):
        for f in (HOST_OUT, HOST_KEY, untagged):
            if os.path.exists(f):
                os.remove(f)
        print("host path not built: %s" % why, file=sys.stderr)

    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return not_built("no torch")
    torch_dir = list(spec.submodule_search_locations)[0]
    try:
        key = host_key(_torch_version(torch_dir))
        if not force and os.path.exists(HOST_OUT) and os.path.exists(HOST_KEY):
            with open(HOST_KEY) as f:
                if f.read() == key:
                    return HOST_OUT
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
        tmp = HOST_OUT + ".tmp%d" % os.getpid()
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", '-DGDN_HOST_KEY="%s"' % key,
               "-I" + os.path.join(torch_dir, "include"),
               "-I" + os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               "-I" + os.path.join(cuda, "include"), "-I" + sysconfig.get_paths()["include"], HOST_SRC, "-o", tmp,
               "-L" + os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            return not_built("\n" + r.stderr[-4000:])
        if os.path.exists(untagged):
            os.remove(untagged)
        os.replace(tmp, HOST_OUT)
        os.makedirs(os.path.dirname(HOST_KEY), exist_ok=True)
        with open(HOST_KEY, "w") as f:
            f.write(key)
    except (OSError, AttributeError, RuntimeError) as e:
        return not_built(e)
    return HOST_OUT


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "host.cpp"] + [os.path.join(ROOT, "include", "gdn.h"),
                                                                  __file__]
    return max(os.path.getmtime(f) for f in files)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    out = build_library(force, verbose, extra)
    build_host(force)
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
