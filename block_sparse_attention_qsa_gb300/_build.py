"""Builds libqsa.so in-tree for sm_103a with nvcc (no cmake, no torch build).

Each .cu under csrc/ compiles to an object in parallel; the objects link into
``block_sparse_attention_qsa_gb300/libqsa.so`` with the CUDA runtime linked
statically, so the library only needs the NVIDIA driver at run time.

The binding's fast path (csrc/qsa_fast.cpp, the module ``_fast``) compiles
beside them with g++ against the headers of this Python and this torch, whose
versions are in its file's name: another Python or torch never loads it, and
builds its own. The binding works without it (its calls take a few microseconds
more on the host), so where it cannot be compiled the build warns and goes on.

``build(trace=True)`` makes the tracing build instead, ``libqsa_trace.so``
(the same sources with ``-DQSA_TRACE``: the step's kernels record per-CTA
phase stamps, read back with ``qsa_trace_read``); ``timeline.py`` uses it.
"""

from __future__ import annotations

import concurrent.futures
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libqsa.so")
BUILD_TRACE = os.path.join(PKG, "_build_trace")
LIB_TRACE = os.path.join(PKG, "libqsa_trace.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the QSA library needs the CUDA toolkit to build")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def fast_path() -> str:
    """The file of the module ``_fast`` for the running Python and torch."""
    import torch

    return os.path.join(PKG, f"_fast.torch-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _newest_input() -> float:
    files = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h", ".cpp"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def _fast_cmd(out: str):
    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    # torch's libraries are found by name in the process that imported torch
    return [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-isystem", inc,
            os.path.join(CSRC, "qsa_fast.cpp"), "-o", out, "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10"]


def check_registers(log: str) -> int:
    """Raises where the compiler's report has a prefix_kernel whose registers are
    not those that its warpgroups share out: a thread's part of 65,536, in steps
    of 8. Its setmaxnreg would wait for registers that the launch does not have
    (the library refuses such a launch, with no more than a CUDA error). Kernels of
    up to 256 threads share nothing out. Returns the kernels seen."""
    seen, kernel = 0, None
    for line in log.splitlines():
        entry = re.search(r"Compiling entry function '(\w+)'", line)
        if entry:  # prefix_kernel<Pc<head dim, E4M3, row tiles>>
            kernel = re.search(r"prefix_kernelI\w*?2PcILi(\d+)ELb([01])ELi(\d+)E", entry.group(1))
        used = re.search(r"Used (\d+) registers", line)
        if used and kernel:
            seen += 1
            threads = 128 * (int(kernel.group(3)) + int(kernel.group(2)) + 1)
            want = 65536 // threads // 8 * 8
            if threads > 256 and int(used.group(1)) != want:
                raise RuntimeError(
                    f"prefix_kernel of head dim {kernel.group(1)}, {'E4M3' if kernel.group(2) == '1' else 'BF16'}, "
                    f"{kernel.group(3)} row tiles: {used.group(1)} registers a thread, its warpgroups share out {want}: "
                    "this compiler needs other shares (kSoftRegs, kOtherRegs in qsa_prefix.cuh)")
            kernel = None
    return seen


def build(force: bool = False, verbose: bool = False, extra_flags=(), trace: bool = False) -> str:
    """Compile and link libqsa.so (or, with ``trace``, libqsa_trace.so), and
    the fast path's module; returns the library's path. Of the two, what is
    newer than every source is left as it is unless ``force``."""
    lib, bdir = (LIB_TRACE, BUILD_TRACE) if trace else (LIB, BUILD)
    if trace:
        extra_flags = (*extra_flags, "-DQSA_TRACE")
    newest = _newest_input()

    def stale(path):
        return force or not os.path.exists(path) or os.path.getmtime(path) < newest

    fast = fast_path()
    make_lib, make_fast = stale(lib), stale(fast)
    cmds, objs = [], []
    if make_lib:
        os.makedirs(bdir, exist_ok=True)
        cc = nvcc()
        for src in sources():
            obj = os.path.join(bdir, os.path.basename(src)[:-3] + ".o")
            objs.append(obj)
            report = ["-Xptxas", "-v"] if os.path.basename(src).startswith("qsa_prefix") else []
            cmds.append([cc, *ARCH, *FLAGS, *report, *extra_flags, "-c", src, "-o", obj])

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compiler failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return r.stderr

    def run_fast():
        try:
            run(_fast_cmd(fast + ".tmp"))
            os.replace(fast + ".tmp", fast)
        except (OSError, RuntimeError) as e:
            warnings.warn(f"the binding's fast path was not built, it works without: {e}", RuntimeWarning)

    with concurrent.futures.ThreadPoolExecutor(max_workers=10) as ex:
        made_fast = ex.submit(run_fast) if make_fast else None
        logs = list(ex.map(run, cmds))
        if made_fast:
            made_fast.result()
    if make_lib and check_registers("\n".join(logs)) == 0:
        warnings.warn("the compiler's report names no prefix_kernel: its registers were not checked", RuntimeWarning)
    if verbose:
        for lg in logs:
            if lg.strip():
                print(lg)
    if make_lib:
        tmp = lib + ".tmp"
        run([cc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else []
    print(build(force=True, verbose=v or bool(extra), extra_flags=extra))
