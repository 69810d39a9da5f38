"""Build libdkv.so in-tree with nvcc for sm_100a.

    python decode_attention_host_b200/build.py [--verbose]

Run it by path: importing the package itself needs the built library.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
LIB = PKG / "libdkv.so"
SOURCES = [CSRC / "dkv_api.cu", CSRC / "dkv_noalloc.cu", CSRC / "dkv_serve.cu", CSRC / "dkv_host.cpp"]
HEADERS = [CSRC / "dkv_kernels.cuh", CSRC / "dkv_append.cuh", CSRC / "dkv_multi.cuh", CSRC / "dkv_chunk.cuh",
           CSRC / "dkv_tables.cuh", CSRC / "dkv_handle.h", CSRC / "dkv_error.h", CSRC / "dkv_plan.h",
           CSRC / "dkv_tma.h", ROOT / "include" / "dkv.h"]
# named with this Python's ABI tag, so that another Python never loads it
CALL_LIB = PKG / ("_dkv_call" + sysconfig.get_config_var("EXT_SUFFIX"))
CALL_SOURCE = CSRC / "dkv_python.cpp"
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "-shared", "-cudart", "static",
         f"-I{ROOT / 'include'}", f"-I{CSRC}"]


def up_to_date() -> bool:
    return LIB.exists() and all(p.stat().st_mtime <= LIB.stat().st_mtime for p in SOURCES + HEADERS + [Path(__file__)])


def build_calls(force: bool = False) -> Path | None:
    """Compile the CPython calls (host code only; they open libdkv.so at import).  Without Python's headers there are
    none, and the package makes the same calls through ctypes."""
    (PKG / "_dkv_call.so").unlink(missing_ok=True)   # an untagged build, which any Python would load
    if not (Path(sysconfig.get_paths()["include"]) / "Python.h").exists():
        print("no Python.h: the serving step's calls go through ctypes", file=sys.stderr)
        return None
    newest = max(p.stat().st_mtime for p in (CALL_SOURCE, ROOT / "include" / "dkv.h", Path(__file__)))
    if force or not CALL_LIB.exists() or CALL_LIB.stat().st_mtime < newest:
        tmp = CALL_LIB.with_suffix(f".{os.getpid()}.tmp.so")
        subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-fPIC", "-fvisibility=hidden", "-shared",
                        f"-I{sysconfig.get_paths()['include']}", f"-I{ROOT / 'include'}", "-o", str(tmp),
                        str(CALL_SOURCE), "-ldl"], check=True)
        os.replace(tmp, CALL_LIB)
    return CALL_LIB


def build(force: bool = False, verbose: bool = False, out: Path = LIB, defines: tuple[str, ...] = ()) -> Path:
    """Compile the library to ``out``; ``defines`` are extra -D build-time knobs (e.g. DKV_DEV_STAGES=2)."""
    out = Path(out)
    if not force and not defines and out == LIB and up_to_date():
        build_calls()
        return LIB
    tmp = out.with_suffix(f".{os.getpid()}.tmp.so")
    cmd = [NVCC, *FLAGS, *(f"-D{d}" for d in defines), *(["-Xptxas", "-v"] if verbose else []), "-o", str(tmp),
           *map(str, SOURCES)]
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)
    build_calls(force)
    return out


if __name__ == "__main__":
    args = sys.argv[1:]
    out = Path(args[args.index("--out") + 1]) if "--out" in args else LIB
    defines = tuple(a[2:] for a in args if a.startswith("-D"))
    print(build(force=True, verbose="--verbose" in args, out=out, defines=defines))
