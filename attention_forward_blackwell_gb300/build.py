"""Builds libfa_gb300.so from csrc/ with nvcc for sm_103a (in-tree), and
_bind, the Python module of the serving operators, from csrc/bind.cpp (where torch
is installed: the library itself needs none).

Each translation unit is compiled in parallel into ``_build/`` and the objects
are linked into ``libfa_gb300.so`` next to this file.  Objects are rebuilt
when their source or any header is newer.
"""
from __future__ import annotations

import importlib.util
import os
import platform
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OBJDIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libfa_gb300.so")
BIND_PATH = os.path.join(HERE, "_bind" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["prefill_d512.cu", "prefill_d128.cu", "prefill_d256.cu", "prefill_d96.cu",
           "prefill_d64.cu", "decode.cu", "selftest.cu", "api.cu", "decode_noalloc.cu", "cache.cu",
           "span.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
                "-I", CSRC, "-I", INCLUDE]


def _options():
    """Build options from the environment: FA_PREFILL_TRACE=1 compiles the
    prefill kernel's debug clock trace (off by default: it costs registers)."""
    return ["-DFA_PREFILL_TRACE=1"] if os.environ.get("FA_PREFILL_TRACE") == "1" else []


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _torch():
    """Folder of the installed torch package and its version; None, None without torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None, None
    root = os.path.dirname(spec.origin)
    about = {}
    with open(os.path.join(root, "version.py")) as f:
        exec(f.read(), about)
    return root, about["__version__"]


def _cuda_home():
    nvcc = _nvcc()
    nvcc = os.path.realpath(nvcc) if os.path.sep in nvcc else "/usr/local/cuda/bin/nvcc"
    return os.path.dirname(os.path.dirname(nvcc))


def _compile_bind(force):
    """csrc/bind.cpp against the installed torch."""
    src, obj = os.path.join(CSRC, "bind.cpp"), os.path.join(OBJDIR, "bind.o")
    newest = max(os.path.getmtime(src), os.path.getmtime(os.path.join(INCLUDE, "fa.h")))
    if not force and os.path.exists(obj) and os.path.getmtime(obj) >= newest:
        return
    include = os.path.join(_torch()[0], "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-c", src, "-o", obj + ".tmp",
           "-I", include, "-I", os.path.join(include, "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(_cuda_home(), "include")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for bind.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(obj + ".tmp", obj)


def _link_bind():
    libs = os.path.join(_torch()[0], "lib")
    tmp = BIND_PATH + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, os.path.join(OBJDIR, "bind.o"),
           LIB_PATH, "-L", libs, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND_PATH)


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    hs.append(os.path.join(INCLUDE, "fa.h"))
    return hs


def build(force: bool = False, jobs: int | None = None, verbose: bool = False) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    with_bind = _torch()[0] is not None
    # objects for another host architecture, Python or torch are never reused
    stamp = os.path.join(OBJDIR, "host.txt")
    host = (f"{platform.machine()} {platform.system()} {sysconfig.get_config_var('SOABI')} "
            f"torch {_torch()[1]} {' '.join(_options())}")
    if not os.path.exists(stamp) or open(stamp).read() != host:
        force = True
    nvcc = _nvcc()
    newest_header = max(os.path.getmtime(h) for h in _headers())

    def compile_one(src):
        s = os.path.join(CSRC, src)
        o = os.path.join(OBJDIR, src.replace(".cu", ".o"))
        if (not force and os.path.exists(o)
                and os.path.getmtime(o) >= max(os.path.getmtime(s), newest_header)):
            return o, False
        cmd = [nvcc] + FLAGS + _options() + ["-c", s, "-o", o + ".tmp"]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        os.replace(o + ".tmp", o)
        return o, True

    jobs = jobs or min(len(SOURCES), os.cpu_count() or 4)
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        bind = ex.submit(_compile_bind, force) if with_bind else None
        results = list(ex.map(compile_one, SOURCES))
        if bind is not None:
            bind.result()
    # (by age, as the library: an earlier build may have failed after bind.o)
    relink_bind = with_bind and (
        not os.path.exists(BIND_PATH)
        or os.path.getmtime(BIND_PATH) < os.path.getmtime(os.path.join(OBJDIR, "bind.o")))
    objs = [o for o, _ in results]
    relink = (force or any(changed for _, changed in results) or not os.path.exists(LIB_PATH)
              or os.path.getmtime(LIB_PATH) < max(os.path.getmtime(o) for o in objs))
    if relink:
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs + [
            "-Xlinker", "-soname=libfa_gb300.so",
            "-Xlinker", "-rpath," + os.path.join(_cuda_home(), "lib64")]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        # a module of other arguments is never left beside the new library
        if relink_bind and os.path.exists(BIND_PATH):
            os.remove(BIND_PATH)
        os.replace(tmp, LIB_PATH)
    if relink_bind:
        _link_bind()
    with open(stamp, "w") as f:
        f.write(host)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
