"""Builds libkvevict.so in-tree with nvcc for sm_103a (no torch extension machinery)."""
from __future__ import annotations

import concurrent.futures
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
LIB = os.path.join(PKG, "libkvevict.so")
FAST = os.path.join(PKG, "_fast.so")   # the Python binding's common case (csrc/binding.cpp),
STAMP = os.path.join(BUILD, "binding.txt")   # and the torch and Python that it was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
                     "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    return (glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)])


def _stale(target: str, inputs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in inputs)


def binding_tag() -> str:
    """The torch and the Python at hand: _fast.so reads tensors by their layout in one of each."""
    import torch
    return "%s %s %s" % (torch.__version__, sys.version, os.path.dirname(torch.__file__))


def binding_built_for() -> str:
    """The tag that _fast.so was built for, empty where that is not known."""
    if not os.path.exists(STAMP):
        return ""
    with open(STAMP) as f:
        return f.read()


def _no_fast(why: str) -> None:
    print("kv_cache_eviction_gb300: no _fast.so (calls go through ctypes): %s" % why,
          file=sys.stderr)
    if os.path.exists(FAST):
        os.remove(FAST)


def _build_fast() -> None:
    """Compile csrc/binding.cpp against the torch at hand.  Without it (no Python or torch headers,
    no g++) calls go through ctypes, 6 us slower each: said, not raised."""
    src = os.path.join(CSRC, "binding.cpp")
    try:
        import torch
    except ImportError:
        return
    except Exception as e:   # (a torch whose libraries do not load: OSError, RuntimeError)
        _no_fast("torch does not load: %s" % e)
        return
    tag = binding_tag()
    if binding_built_for() == tag and not _stale(FAST, [src] + _deps()):
        return
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc.append(os.path.join(cuda, "include"))
    tmp = FAST + ".tmp"
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden"] +
           ["-I" + x for x in inc] + [src, "-o", tmp, "-L" + os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"])
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = "" if r.returncode == 0 else r.stderr[-2000:]
    except OSError as e:
        why = str(e)
    if why:
        _no_fast(why)
        return
    if os.path.exists(STAMP):   # (never an old tag beside a new module, wherever this is cut short)
        os.remove(STAMP)
    os.replace(tmp, FAST)
    with open(STAMP, "w") as f:
        f.write(tag)


def build(verbose: bool = False, jobs: int = 0) -> str:
    """Compile every .cu under csrc/ in parallel and link libkvevict.so. Returns its path."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = _deps()
    todo = []
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if _stale(o, [s] + deps):
            todo.append((s, o))

    def compile_one(so):
        s, o = so
        cmd = [nvcc] + NVCC_FLAGS + ["-c", s, "-o", o]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s%s" % (s, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return o

    n = jobs or min(len(todo) + 1, os.cpu_count() or 4)
    with concurrent.futures.ThreadPoolExecutor(max_workers=n) as ex:
        fast = ex.submit(_build_fast)
        list(ex.map(compile_one, todo))
        fast.result()
    if todo or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
