"""Builds the HIP libraries for gfx950 with hipcc, in-tree: libcp.so (the
lookup library, include/cp.h and include/cp_ops.h), libcp_probe.so (measurement
probes, include/cp_probe.h) and _cp_torch.so (the dense operators' functions on
torch tensors, host code on top of libcp.so)."""
from __future__ import annotations

import hashlib
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SOURCES = [os.path.join(CSRC, "cp_decode.hip"), os.path.join(CSRC, "cp_dedup.hip"),
           os.path.join(CSRC, "cp_encode.hip"), os.path.join(CSRC, "cp_mixed.hip"),
           os.path.join(CSRC, "cp_shard.hip"), os.path.join(CSRC, "cp_dedup_mixed.hip"),
           os.path.join(CSRC, "cp_api.hip"),
           os.path.join(CSRC, "cp_embed.hip"), os.path.join(CSRC, "cp_norm.hip"), os.path.join(CSRC, "cp_quant.hip"),
           os.path.join(CSRC, "cp_gemm.hip"), os.path.join(CSRC, "cp_ops_api.hip"),
           os.path.join(CSRC, "cp_linear.hip"), os.path.join(CSRC, "cp_linear_dx.hip"),
           os.path.join(CSRC, "cp_linear_dw.hip"), os.path.join(CSRC, "cp_dropout.hip"),
           os.path.join(CSRC, "cp_linear_api.hip")]
DEPS = SOURCES + [os.path.join(CSRC, "cp_internal.h"), os.path.join(CSRC, "cp_lane.h"),
                  os.path.join(CSRC, "cp_encode_copies.h"),
                  os.path.join(CSRC, "cp_status.h"), os.path.join(CSRC, "cp_ops_internal.h"),
                  os.path.join(CSRC, "cp_linear_internal.h"), os.path.join(CSRC, "cp_linear_tile.h"),
                  os.path.join(ROOT, "include", "cp.h"), os.path.join(ROOT, "include", "cp_ops.h"),
                  os.path.join(ROOT, "include", "cp_linear.h")]
LIB = os.path.join(PKG, "libcp.so")
PROBE_SOURCES = [os.path.join(CSRC, "cp_probe.hip")]
PROBE_LIB = os.path.join(PKG, "libcp_probe.so")
TORCH_SOURCES = [os.path.join(CSRC, "cp_torch.cpp"), os.path.join(CSRC, "cp_torch_linear.cpp")]
TORCH_LIB = os.path.join(PKG, "_cp_torch.so")
TORCH_DEPS = TORCH_SOURCES + [os.path.join(CSRC, "cp_torch.h"), os.path.join(ROOT, "include", "cp.h"),
                              os.path.join(ROOT, "include", "cp_ops.h"), os.path.join(ROOT, "include", "cp_linear.h")]
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    # no packed fp32 math: keep float code on plain (scalar-lane) instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-parameter", "-Wundef",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    return "hipcc"


def is_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in DEPS)


def _hipcc(sources: list[str], lib: str, verbose: bool, extra_flags: list[str] | None) -> str:
    """One object a source, several at a time, and the library from them."""
    tmp = lib + ".tmp%d" % os.getpid()
    flags = [*HIPCC_FLAGS, *(extra_flags or []), "-I", os.path.join(ROOT, "include")]
    with tempfile.TemporaryDirectory() as folder, ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        objects = [os.path.join(folder, os.path.basename(s) + ".o") for s in sources]
        list(pool.map(lambda pair: _compile([hipcc(), *flags, "-c", pair[0], "-o", pair[1]], lib, verbose),
                      zip(sources, objects)))
        return _run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objects, "-o", tmp], tmp, lib, verbose)


def _compile(cmd: list[str], lib: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed building {os.path.basename(lib)}")


def _run(cmd: list[str], tmp: str, lib: str, verbose: bool) -> str:
    _compile(cmd, lib, verbose)
    os.replace(tmp, lib)
    return lib


def build(verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Builds the libraries; returns the path of libcp.so."""
    _hipcc(PROBE_SOURCES, PROBE_LIB, verbose, extra_flags)
    lib = _hipcc(SOURCES, LIB, verbose, extra_flags)
    build_torch(verbose)
    return lib


def _torch_folder() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]  # without importing it


def _torch_mark() -> str:
    """What _cp_torch.so carries of the torch it was built for."""
    with open(os.path.join(_torch_folder(), "version.py")) as f:
        version = re.search(r"__version__ = '([^']*)'", f.read()).group(1)
    return f"[built for torch {version}]"


def _source_mark() -> str:
    """What it carries of its sources."""
    digest = hashlib.sha256()
    for path in TORCH_DEPS:
        with open(path, "rb") as f:
            digest.update(f.read())
    return f"[built from {digest.hexdigest()[:16]}]"


def torch_built() -> tuple[bool, bool]:
    """Whether _cp_torch.so is there, built for the torch that is installed,
    and whether it is built from the present sources (where there are any)."""
    if not os.path.exists(TORCH_LIB):
        return False, False
    with open(TORCH_LIB, "rb") as f:
        held = f.read()
    sources = all(os.path.exists(p) for p in TORCH_DEPS)
    return _torch_mark().encode() in held, not sources or _source_mark().encode() in held


def build_torch(verbose: bool = False) -> str:
    """Builds _cp_torch.so, a CPython module, against the torch that is
    installed and libcp.so beside it."""
    torch = _torch_folder()
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc()))) if os.path.isabs(hipcc()) else "/opt/rocm"
    include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               os.path.join(rocm, "include"), sysconfig.get_paths()["include"]]
    tmp = TORCH_LIB + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D__HIP_PLATFORM_AMD__=1",  # what hipcc itself defines; the HIP headers ask for it
           '-DCP_TORCH_MARKS="%s"' % " ".join((_torch_mark(), _source_mark())),
           *(x for d in include for x in ("-isystem", d)), *TORCH_SOURCES, "-o", tmp,
           "-L", PKG, "-l:" + os.path.basename(LIB), "-L", os.path.join(torch, "lib"),
           "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    return _run(cmd, tmp, TORCH_LIB, verbose)


if __name__ == "__main__":
    print(build(verbose=True))
