"""Host-only build of the packer and layout (no HIP code) with the address
and undefined-behaviour sanitizers, for the CPU tests.

The tests load it through the SGEMV_LIB variable in a child process whose
LD_PRELOAD starts with the address-sanitizer runtime; any report aborts that
process. The GPU code is never built this way.
"""
import os
import subprocess

from ._build import CSRC, HOST_SRCS, OUT_DIR, _run

SAN_LIB = os.path.join(OUT_DIR, "libsgemv_host_san.so")


def build_host_sanitized(verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    tmp = SAN_LIB + ".tmp"
    _run(["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-shared", "-ffp-contract=off", "-fno-fast-math",
          "-fno-omit-frame-pointer", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
          "-Wall", "-Wextra"] + [os.path.join(CSRC, s) for s in HOST_SRCS] + ["-o", tmp], verbose)
    os.replace(tmp, SAN_LIB)
    return SAN_LIB


def asan_runtime() -> str:
    """Path of the compiler's address-sanitizer runtime (to preload)."""
    return subprocess.run(["g++", "-print-file-name=libasan.so"], stdout=subprocess.PIPE, text=True,
                          check=True).stdout.strip()


# The decode-step operators' index arithmetic (csrc/decode_index.hpp, shared
# with the kernels) as programs of their own for the CPU tests.
_INDEX_DIR = os.path.join(os.path.dirname(os.path.dirname(CSRC)), "tests", "decode_index")
INDEX_SRC = os.path.join(_INDEX_DIR, "index_check.cpp")
INDEX_CHECK = os.path.join(_INDEX_DIR, "_build", "index_check")
VISIBLE_SRC = os.path.join(_INDEX_DIR, "visible_check.cpp")
VISIBLE_CHECK = os.path.join(_INDEX_DIR, "_build", "visible_check")


def build_index_check(verbose: bool = False) -> str:
    os.makedirs(os.path.dirname(INDEX_CHECK), exist_ok=True)
    for src, exe in ((INDEX_SRC, INDEX_CHECK), (VISIBLE_SRC, VISIBLE_CHECK)):
        tmp = exe + ".tmp"
        _run(["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
              "-fno-sanitize-recover=all", "-Wall", "-Wextra", src, "-o", tmp], verbose)
        os.replace(tmp, exe)
    return INDEX_CHECK
