"""Build step of the C-ABI library ``libspecverify.so`` (sm_103a) and of
``_serve_calls.so``, the serving operators' argument marshalling for Python
(host code over torch's headers, linked to the library).

One translation unit each for the verify step, its vocabulary-sharded form,
slot maps and cache writes, sampling, and paged attention; one ``-gencode``,
compiled in parallel, in-tree next to this file, with ``nvcc -shared``.
Rebuilds only when a source or a header is newer than the library; the calls
also where they were built for another torch or Python.  The verify step needs
the library alone: where the calls cannot be built, that is a warning.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libspecverify.so")
CALLS = os.path.join(HERE, "_serve_calls.so")
CALLS_STAMP = CALLS + ".stamp"  # the torch and Python that the calls were built for
CALLS_SOURCE = os.path.join(CSRC, "serve_calls.cpp")
SOURCES = [os.path.join(CSRC, f) for f in ("spec_verify.cu", "sv_shard.cu", "sv_slots.cu",
                                           "sv_sample.cu", "sv_attention.cu")]
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return files


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libspecverify.so")


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(f) > t for f in deps)


def _run(tool, cmd, verbose):
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{tool} failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    if verbose:
        print(res.stdout + res.stderr)


def calls_stamp() -> str:
    """The torch and Python of this process, whose binary interfaces the calls need."""
    import sysconfig

    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def calls_built_for():
    """What the built calls need, None where that is not recorded."""
    if not os.path.exists(CALLS_STAMP):
        return None
    with open(CALLS_STAMP) as f:
        return f.read()


def _build_calls(verbose: bool) -> None:
    import sysconfig

    import torch
    for old in (CALLS, CALLS_STAMP):  # not left beside another library
        if os.path.exists(old):
            os.remove(old)
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    inc = [os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    lib = os.path.join(root, "lib")
    _run("g++", ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", INCLUDE,
                 *[x for i in inc for x in ("-isystem", i)],
                 f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                 CALLS_SOURCE, "-o", CALLS + ".tmp", LIB, f"-L{lib}", "-ltorch_python", "-ltorch",
                 "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-Wl,-rpath,$ORIGIN:{lib}"], verbose)
    os.replace(CALLS + ".tmp", CALLS)
    with open(CALLS_STAMP, "w") as f:
        f.write(calls_stamp())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is out of date; returns the path of libspecverify.so."""
    if force or _stale(LIB, _deps()):
        _run("nvcc", [nvcc_path(), ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared", "--threads", "0",
                      "-Xcompiler", "-fPIC", "-Xptxas", "-v" if verbose else "-O3",
                      "-Xlinker", "-soname=libspecverify.so",
                      "-I", INCLUDE, "-I", CSRC, *SOURCES, "-o", LIB + ".tmp", "-lcudart"], verbose)
        os.replace(LIB + ".tmp", LIB)
    if force or _stale(CALLS, [CALLS_SOURCE, LIB]) or calls_built_for() != calls_stamp():
        try:
            _build_calls(verbose)
        except (ImportError, OSError, RuntimeError) as e:
            warnings.warn(f"the serving operators' Python calls were not built: {e}")
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
