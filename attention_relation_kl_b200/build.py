"""Build librelkl.so in-tree for sm_100a (B200) with nvcc, and the binding's
marshalling module (plain C++ against torch's headers).

    python -m attention_relation_kl_b200.build        # or build() from Python

The library is placed next to this file so that it travels with the source
tree.  nvcc cross-compiles without a GPU.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "librelkl.so")
SOURCES = ["relkl_api.cu", "relkl_tc.cu", "relkl_simt.cu", "relkl_chain.cu", "relkl_gemm.cu",
           "relkl_rotary.cu", "relkl_adamw.cu", "relkl_int8.cu"]
HEADERS = ["relkl_device.cuh", "relkl_params.h", "relkl_ranges.h"]
MARSHAL_SOURCE = os.path.join(CSRC, "relkl_marshal.cpp")
MARSHAL = os.path.join(HERE, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-cudart", "static",
]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    deps.append(os.path.join(ROOT, "include", "relkl.h"))
    deps.append(__file__)
    return any(os.path.getmtime(p) > t for p in deps)


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")


def _torch() -> str:
    """Which torch is installed, without importing it: its version, and where it is."""
    where = importlib.util.find_spec("torch").submodule_search_locations[0]
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "unknown"
    return f"{version} {where}"


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    """Compile the marshalling module if its sources are newer, or if it was built for
    another torch (which stands in a file beside it); returns its path."""
    deps = [MARSHAL_SOURCE, os.path.join(CSRC, "relkl_ranges.h"), os.path.join(ROOT, "include", "relkl.h"),
            __file__]
    record, torch_now = MARSHAL + ".torch", _torch()
    if not force and os.path.exists(MARSHAL) and os.path.exists(record) and \
            all(os.path.getmtime(p) <= os.path.getmtime(MARSHAL) for p in deps):
        with open(record) as f:
            if f.read() == torch_now:
                return MARSHAL
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    inc, lib = os.path.join(torch_dir, "include"), os.path.join(torch_dir, "lib")
    tmp = MARSHAL + ".tmp"
    _run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", inc,
          "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
          "-I", sysconfig.get_paths()["include"], MARSHAL_SOURCE, "-L", lib, f"-Wl,-rpath,{lib}",
          "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-o", tmp], verbose)
    os.replace(tmp, MARSHAL)
    with open(record, "w") as f:
        f.write(torch_now)
    return MARSHAL


def build(force: bool = False, verbose: bool = False, checks: bool = False) -> str:
    """Compile librelkl.so if any source is newer; returns its path.  Then the
    marshalling module, which needs Python's and torch's headers: where it cannot be
    compiled there is a warning, and the loss, which does without, can be used.

    ``checks`` (or RELKL_CHECKS=1 in the environment) builds the debug variant
    that replays every tensor-core launch's schedule on the host first
    (relkl_check_schedule) and refuses a launch whose schedule is unsound."""
    checks = checks or os.environ.get("RELKL_CHECKS") == "1"
    if force or checks or _stale():
        tmp = LIB + ".tmp"
        cmd = [nvcc_path(), *NVCC_FLAGS, *(["-DRELKL_CHECKS"] if checks else []),
               "-I", os.path.join(ROOT, "include"),
               *[os.path.join(CSRC, f) for f in SOURCES], "-ldl", "-o", tmp]
        _run(cmd, verbose)
        os.replace(tmp, LIB)
    try:
        build_marshal(force, verbose)
    except Exception as e:     # the library is whole without it; an old one may not fit it
        if os.path.exists(MARSHAL):
            os.remove(MARSHAL)
        warnings.warn(f"the operators that need the marshalling module cannot be called: {e}")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, checks="--checks" in sys.argv))
