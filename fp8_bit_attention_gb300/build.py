"""Build libovc (the C ABI in include/ovc.h) in-tree for sm_103a with nvcc."""
from __future__ import annotations

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SRCS = [os.path.join(CSRC, f) for f in ("ovc.cu", "paged.cu", "serve.cu")]
HEADERS = [os.path.join(CSRC, f) for f in ("ptx.cuh", "prepare.cuh", "attention.cuh", "repair.cuh", "group.cuh",
                                           "host_stream.cuh", "host.cuh", "paged.cuh", "paged_plan.cuh",
                                           "paged_decode.cuh", "paged_chunk.cuh", "paged_args.cuh", "pages.cuh", "move.cuh",
                                           "drafts.cuh")]
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD_DIR, "libovc.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def compile_command(src: str, out: str) -> list[str]:
    return ["nvcc", "-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-c", "-o", out, src]


def link_command(objs: list[str], out: str) -> list[str]:
    return ["nvcc", *ARCH, "-shared", "-o", out, *objs]


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [*SRCS, os.path.join(INCLUDE, "ovc.h"), *HEADERS]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libovc.so (skipped when up to date; the translation units in
    parallel) and return its path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    if not force and not _stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    objs = [f"{tmp}.{os.path.basename(s)}.o" for s in SRCS]
    cmds = [compile_command(s, o) for s, o in zip(SRCS, objs)]
    link = link_command(objs, tmp)
    if verbose:
        for cmd in (*cmds, link):
            print(" ".join(cmd))
    try:
        with ThreadPoolExecutor(len(cmds)) as ex:
            for f in [ex.submit(subprocess.run, cmd, check=True) for cmd in cmds]:
                f.result()
        subprocess.run(link, check=True)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
