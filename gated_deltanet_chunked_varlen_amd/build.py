"""Build libgdn_prefill.so in-tree with hipcc for gfx950.

Each source compiles to its own object in parallel, then one link step makes
the shared library.  _calls.so, the CPython module that marshals the
recurrence's and the state pool's calls, is host code against torch's headers.

Usage: python -m gated_deltanet_chunked_varlen_amd.build
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libgdn_prefill.so")
SOURCES = ["gdn_host.hip", "k0_chunk_index.hip", "k1_intra.hip",
           "k2_state.hip", "k3_output.hip", "k4_decode.hip", "k5_cp.hip",
           "gdn_recurrence_host.hip", "k6_recurrence.hip", "k7_pool.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Wall", "-Wno-unused-function",
    # keep packed fp32 instructions out of device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


CALLS = os.path.join(HERE, "_calls.so")
CXX = os.environ.get("CXX", "g++")


def build_calls(verbose: bool = False, out: str = CALLS) -> str:
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    tmp = out + ".tmp%d" % os.getpid()
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)]
    cmd += ["-isystem" + p for p in include_paths() + [sysconfig.get_paths()["include"]]]
    cmd += [os.path.join(CSRC, "torch_calls.cpp"), "-o", tmp]
    cmd += ["-L" + p for p in library_paths()] + ["-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed on torch_calls.cpp:\n%s" % (CXX, r.stderr))
    os.replace(tmp, out)
    return out


def _clean(stderr: str) -> str:
    return "\n".join(l for l in stderr.splitlines() if "packed-fp32-ops" not in l)


def build(verbose: bool = False, extra_flags=None, out: str = LIB) -> str:
    flags = FLAGS + list(extra_flags or [])
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    with tempfile.TemporaryDirectory(prefix="gdn_build_") as tmpdir:
        objs = [os.path.join(tmpdir, os.path.basename(s) + ".o") for s in srcs]

        def compile_one(i):
            cmd = [HIPCC] + flags + ["-c", srcs[i], "-o", objs[i]]
            if verbose:
                print(" ".join(cmd), flush=True)
            return subprocess.run(cmd, capture_output=True, text=True)

        jobs = max(1, min(len(srcs), os.cpu_count() or 1, 16))
        with ThreadPoolExecutor(jobs) as ex:
            results = list(ex.map(compile_one, range(len(srcs))))
        for s, r in zip(srcs, results):
            err = _clean(r.stderr)
            if r.returncode != 0:
                raise RuntimeError("hipcc failed on %s:\n%s" % (os.path.basename(s), err))
            if verbose and err.strip():
                print(err, file=sys.stderr)
        tmp = out + ".tmp%d" % os.getpid()
        cmd = [HIPCC] + flags + ["-shared", "-o", tmp] + objs
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("hipcc link failed:\n" + _clean(r.stderr))
        os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
    print(build_calls(verbose=True))
