"""Build libcowa.so in-tree for sm_100a with nvcc (no GPU needed to build).

    python -m structured_sparse_attention_cowa_b200.build [--debug] [-v]

Compiles every csrc/*.cu to an object in _build/ and links them into
structured_sparse_attention_cowa_b200/libcowa.so (static CUDA runtime; the
driver API is reached through cudaGetDriverEntryPoint, so no -lcuda).
csrc/binding.cpp, the part of the Python binding that is compiled, becomes
_binding.so beside it (against the installed torch; it finds either library's
entry points at run time; without torch it is left out).  Objects are rebuilt only when a source or
header is newer.

--debug builds libcowa_debug.so with COWA_DEBUG=1: the attention kernels check every planned tile
and cache row against the call's tensors before loading it, and a failed check is reported as
COWA_ERR_CHECK through the workspace status (the binding loads this library when the
environment has COWA_DEBUG=1).  The rotary and append kernels have no workspace to report through,
and no checks.
"""

from __future__ import annotations

import argparse
import glob
import hashlib
import importlib.util
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libcowa.so")
LIB_DEBUG = os.path.join(PKG, "libcowa_debug.so")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O3", "--expt-relaxed-constexpr",
          "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _newest_header() -> float:
    hdrs = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    return max((os.path.getmtime(h) for h in hdrs), default=0.0)


def _digest(path: str) -> str:
    with open(path, "rb") as f:
        return hashlib.sha256(f.read()).hexdigest()


def build_binding(verbose: bool = False) -> str:
    """Compile csrc/binding.cpp against the installed torch into _binding.so, if it is out of date: older than
    its sources, or not the file that was last built, or built by another command or against another torch or
    Python (the stamp in _build/ names all of these)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext

    src = os.path.join(CSRC, "binding.cpp")
    hdr = os.path.join(ROOT, "include", "cowa.h")
    stamp = os.path.join(BUILD, "binding.stamp")
    new = BINDING + f".{os.getpid()}.tmp"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))) if os.path.isabs(_nvcc()) else "/usr/local/cuda"
    inc = [*ext.include_paths(), os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *("-isystem" + i for i in inc), src, *("-L" + p for p in ext.library_paths()), "-lc10",
           "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    made_by = "\n".join([torch.__version__, sys.version, *cmd]).replace(ROOT, ".")  # (the tree may be moved)
    if os.path.exists(BINDING) and os.path.exists(stamp) and \
            os.path.getmtime(BINDING) >= max(os.path.getmtime(src), os.path.getmtime(hdr)):
        with open(stamp) as f:
            if f.read() == f"{_digest(BINDING)}\n{made_by}":
                return BINDING
    cmd += ["-o", new]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        if os.path.exists(new):
            os.remove(new)
        raise RuntimeError("g++ failed on binding.cpp")
    digest = _digest(new)
    os.replace(new, BINDING)  # (a program that has the old one loaded keeps it)
    os.makedirs(BUILD, exist_ok=True)
    with open(stamp, "w") as f:
        f.write(f"{digest}\n{made_by}")
    return BINDING


def build(debug: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    flags = list(CFLAGS)
    if debug:
        flags.append("-DCOWA_DEBUG=1")
    if ptxas_info:
        flags += ["-Xptxas", "-v"]
    hdr_t = _newest_header()
    objs, jobs = [], []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + (".dbg.o" if debug else ".o"))
        objs.append(obj)
        if (not ptxas_info and os.path.exists(obj) and os.path.getmtime(obj) >= os.path.getmtime(src)
                and os.path.getmtime(obj) >= hdr_t):
            continue
        jobs.append((src, [nvcc, *ARCH, *flags, "-c", src, "-o", obj]))

    def compile_one(job):
        src, cmd = job
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, r

    # the translation units are independent: compile them side by side
    from concurrent.futures import ThreadPoolExecutor

    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        results = list(ex.map(compile_one, jobs))
    for src, r in results:
        if r.returncode != 0 or verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}")
    out = LIB_DEBUG if debug else LIB
    lib_t = os.path.getmtime(out) if os.path.exists(out) else -1
    if lib_t < max(os.path.getmtime(o) for o in objs):
        cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", out, *objs]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError(f"link of {os.path.basename(out)} failed")
    # after the library, which needs neither torch nor g++
    if importlib.util.find_spec("torch") is None:
        sys.stderr.write("torch is not installed: _binding.so, which only a program with torch can use, is not built\n")
    else:
        build_binding(verbose)
    return out


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--debug", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true")
    args = ap.parse_args()
    print(build(debug=args.debug, verbose=args.verbose, ptxas_info=args.ptxas_info))
