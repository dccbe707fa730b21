"""Build the CUDA library (libpkv_attn.so) in-tree for sm_103a with nvcc, and the Python calls (_binding.so).

Every translation unit under csrc/ is compiled in parallel into _build/, then linked into
libpkv_attn.so next to this file.  Rebuilds only what changed (source or header newer than the
object).  No cmake, no torch extension machinery: the library is a plain C-ABI shared object, and
csrc/python/binding.cpp one host file that is compiled against the headers of Python and torch
(where there is no torch, the library is built alone, for users of its C ABI).
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpkv_attn.so")
BINDING = os.path.join(HERE, "_binding.so")
INCLUDE = os.path.join(ROOT, "include")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")


def _flags(extra=()):
    return ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, "-I", CSRC, *ARCH, *extra]


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(INCLUDE, "*.h"))


def _stale(src, obj, hdr_mtime):
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return os.path.getmtime(src) > t or hdr_mtime > t


def _binding_job(nvcc, force):
    """The command that makes _binding.so; None: it is up to date, or there is no torch, without which nothing could
    import it (the library needs none)."""
    src = os.path.join(CSRC, "python", "binding.cpp")
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    torch = list(spec.submodule_search_locations)[0]
    newest = max(os.path.getmtime(f) for f in (os.path.join(INCLUDE, "pkv_attn.h"), os.path.join(torch, "version.py")))
    if not (force or _stale(src, BINDING, newest)):
        return None
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if not cxx:
        raise RuntimeError("g++ not found (set CXX)")
    lib = os.path.join(torch, "lib")
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(torch, "include"),
           os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")]
    return [cxx, "-std=c++17", "-O2", "-fPIC", "-shared", *("-I" + d for d in inc), "-o", BINDING, src,
            "-L" + lib, "-ltorch_python", "-lc10", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda"]


def build(verbose: bool = False, force: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile csrc/*.cu and csrc/*.cpp for sm_103a and link libpkv_attn.so, compile _binding.so; returns the library's path."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))
    hdr = max([os.path.getmtime(h) for h in _headers()] + [0.0])
    jobs = []
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s) + ".o")
        objs.append(o)
        if force or _stale(s, o, hdr):
            extra = ["-Xptxas", "-v"] if (ptxas_verbose and s.endswith(".cu")) else []
            jobs.append([nvcc, *_flags(extra), "-c", s, "-o", o])

    binding = _binding_job(nvcc, force)
    todo = jobs + ([binding] if binding else [])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    failed = []
    if todo:
        with cf.ThreadPoolExecutor(max_workers=min(len(todo), os.cpu_count() or 4)) as ex:
            for cmd, r in ex.map(run, todo):
                if verbose or ptxas_verbose or r.returncode:
                    print("binding.cpp" if cmd is binding else " ".join(cmd[-3:]), "\n", r.stdout, r.stderr)
                if r.returncode:
                    failed.append("binding.cpp" if cmd is binding else cmd[-3])
    if failed:
        raise RuntimeError("compilation failed for: " + ", ".join(failed))
    newest = max(os.path.getmtime(o) for o in objs)
    if force or jobs or not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        cmd = [nvcc, *ARCH, "-shared", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    return LIB


if __name__ == "__main__":
    import sys

    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv, ptxas_verbose="--ptxas" in sys.argv))
