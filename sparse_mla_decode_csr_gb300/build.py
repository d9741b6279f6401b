"""Build libsmla.so in-tree with nvcc for sm_103a, and _smla.so, its Python calls (no cmake).

Each translation unit under csrc/ compiles in parallel to _build/*.o, then one
link step makes sparse_mla_decode_csr_gb300/libsmla.so from the CUDA sources and
another _smla.so from smla_binding.cpp, which reads PyTorch's tensors and calls
libsmla.so.  Objects are rebuilt only when a source or header is newer than them, the
binding's also when it was made for another Python or PyTorch.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
TRACE = os.environ.get("SMLA_TRACE", "") == "1"  # stage-trace build (debugging only)
BUILD = os.path.join(ROOT, "_build_trace" if TRACE else "_build")
LIB = os.path.join(PKG, "libsmla_trace.so" if TRACE else "libsmla.so")
BINDING = os.path.join(PKG, "_smla.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas=-warn-spills",
              "-I", INCLUDE, "-I", CSRC] + (["-DSMLA_TRACE"] if TRACE else [])


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _torch(*path: str) -> str:
    return os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), *path)


def _made_for(src: str) -> str:
    """What an object is made for besides its sources: the Python and PyTorch whose headers it takes."""
    if src.endswith(".cu"):
        return ""
    with open(_torch("version.py")) as f:
        return f"{sysconfig.get_config_var('SOABI')}\n{_torch()}\n{f.read()}"


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    if any(os.path.getmtime(f) > t for f in [src] + _headers()):
        return True
    what, stamp = _made_for(src), obj + ".for"
    if not what:
        return False
    if not os.path.exists(stamp):
        return True
    with open(stamp) as f:
        return f.read() != what


def _run(cmd, what: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
    if _stale(obj, src):
        if src.endswith(".cu"):
            cmd = [nvcc()] + ARCH + NVCC_FLAGS
        else:
            include = [INCLUDE, _torch("include"), _torch("include", "torch", "csrc", "api", "include"),
                       sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
            cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden"] + \
                [x for d in include for x in ("-isystem" if d != INCLUDE else "-I", d)]
        _run(cmd + ["-c", src, "-o", obj], f"compiling {src}", verbose)
        if _made_for(src):
            with open(obj + ".for", "w") as f:
                f.write(_made_for(src))
    return obj


def _link(out: str, objs, cmd, verbose: bool, force: bool, libs=()) -> None:
    if force or not os.path.exists(out) or any(os.path.getmtime(o) > os.path.getmtime(out) for o in objs):
        _run(cmd + ["-o", out + ".tmp", *objs, *libs], f"linking {out}", verbose)
        os.replace(out + ".tmp", out)


def build(verbose: bool = False, force: bool = False) -> str:
    """Compile every source and link libsmla.so and _smla.so; returns the former's path."""
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu"))) + ([] if TRACE else [os.path.join(CSRC, "smla_binding.cpp")])
    if force:
        for f in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(f)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(sources), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), sources))
    cuda = [o for s, o in zip(sources, objs) if s.endswith(".cu")]
    _link(LIB, cuda, [nvcc()] + ARCH + ["-shared", "-cudart", "shared"], verbose, force)
    if not TRACE:
        # (libraries go behind the object that needs them)
        libs = [f"-L{PKG}", "-Wl,-rpath,$ORIGIN", f"-L{_torch('lib')}", "-l:libsmla.so", "-ltorch_python", "-ltorch_cpu",
                "-lc10", "-lc10_cuda"]
        _link(BINDING, [o for o in objs if o not in cuda], ["g++", "-shared"], verbose, force, libs)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
