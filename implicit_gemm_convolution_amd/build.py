"""Build libigc.so (the HIP kernels and the C ABI) in-tree with hipcc for gfx950,
and, where torch is installed, _marshal.so (the Python binding's marshalling,
host code only) with g++.

The C ABI (csrc/igc.hip, csrc/ffn.hip, csrc/rows.hip, csrc/i8.hip) and the kernel instantiations
(csrc/igc_launch.hip, csrc/ffn_launch.hip and csrc/i8_launch.hip, compiled once
per kernel kind with -DIGC_LAUNCH_UNIT=<n>, -DIGC_FFN_UNIT=<n> and -DIGC_I8_UNIT=<n>) are separate objects
compiled in parallel, then linked into one shared library.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_PATH = os.path.join(PKG, "libigc.so")
ABI_SOURCE = os.path.join(CSRC, "igc.hip")
LAUNCH_SOURCE = os.path.join(CSRC, "igc_launch.hip")
LAUNCH_UNITS = 38  # the (kind, variant) pairs of IGC_LAUNCH_KINDS in igc_host.hpp
FFN_SOURCE = os.path.join(CSRC, "ffn.hip")
FFN_LAUNCH_SOURCE = os.path.join(CSRC, "ffn_launch.hip")
FFN_LAUNCH_UNITS = 10  # the (type, layout) pairs of IGC_FFN_KINDS in ffn_host.hpp, and both types' joint backward launch
ROWS_SOURCE = os.path.join(CSRC, "rows.hip")
I8_SOURCE = os.path.join(CSRC, "i8.hip")
I8_LAUNCH_SOURCE = os.path.join(CSRC, "i8_launch.hip")
I8_LAUNCH_UNITS = 4  # the (output type, layout) pairs of IGC_I8_KINDS in ffn_host.hpp
MARSHAL_SOURCE = os.path.join(CSRC, "marshal.cpp")
MARSHAL_PATH = os.path.join(PKG, "_marshal.so")
SOURCES = [ABI_SOURCE, LAUNCH_SOURCE, FFN_SOURCE, FFN_LAUNCH_SOURCE, ROWS_SOURCE, I8_SOURCE, I8_LAUNCH_SOURCE]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

HIP_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # Every fp32 multiply and add in the epilogues is its own rounded
    # operation: the requantize step is defined with two roundings.
    "-ffp-contract=off",
    # No packed-fp32 instructions anywhere.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def _units():
    """(source, extra defines, object name) of every object of the library."""
    yield ABI_SOURCE, [], "igc.o"
    for n in range(LAUNCH_UNITS):
        yield LAUNCH_SOURCE, [f"-DIGC_LAUNCH_UNIT={n}"], f"igc_launch_{n}.o"
    yield FFN_SOURCE, [], "ffn.o"
    yield ROWS_SOURCE, [], "rows.o"
    for n in range(FFN_LAUNCH_UNITS):
        yield FFN_LAUNCH_SOURCE, [f"-DIGC_FFN_UNIT={n}"], f"ffn_launch_{n}.o"
    yield I8_SOURCE, [], "i8.o"
    for n in range(I8_LAUNCH_UNITS):
        yield I8_LAUNCH_SOURCE, [f"-DIGC_I8_UNIT={n}"], f"i8_launch_{n}.o"


def _jobs() -> int:
    try:
        n = len(os.sched_getaffinity(0))
    except AttributeError:
        n = os.cpu_count() or 1
    return max(1, min(n, 16, LAUNCH_UNITS + 1))


def marshal_command(out: str) -> list | None:
    """The command that compiles _marshal.so against the installed Python and torch; None without torch."""
    try:
        import torch
        from torch.utils import cpp_extension
    except ImportError:
        return None

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + sysconfig.get_paths()["include"],
            *("-I" + p for p in cpp_extension.include_paths()), MARSHAL_SOURCE, "-o", out,
            "-L" + libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10"]


def build(verbose: bool = False, extra_flags=()) -> str:
    """Compile every source; libigc.so and (where torch is installed) _marshal.so go next to this file.  Returns libigc.so's path."""
    tmpdir = tempfile.mkdtemp(prefix="igc_build_")
    try:
        marshal = os.path.join(tmpdir, "_marshal.so")
        extension = marshal_command(marshal)
        cmds = [extension] if extension else []  # (among the longest: first)
        for src, defs, obj in _units():
            cmds.append([HIPCC, *HIP_FLAGS, *extra_flags, *defs, "-c", src, "-o", os.path.join(tmpdir, obj)])

        def run(cmd):
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.check_call(cmd)

        with ThreadPoolExecutor(_jobs()) as ex:
            list(ex.map(run, cmds))
        tmp = LIB_PATH + ".tmp"
        objs = [os.path.join(tmpdir, obj) for _, _, obj in _units()]
        link = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
        run(link)
        os.replace(tmp, LIB_PATH)
        if extension:
            shutil.copyfile(marshal, MARSHAL_PATH + ".tmp")
            os.replace(MARSHAL_PATH + ".tmp", MARSHAL_PATH)
    finally:
        shutil.rmtree(tmpdir, ignore_errors=True)
    return LIB_PATH


def _assembly(out_dir, name, source, define, units, extra_flags):
    os.makedirs(out_dir, exist_ok=True)

    def one(n):
        d = os.path.join(out_dir, f"unit{n}")
        os.makedirs(d, exist_ok=True)
        cmd = [HIPCC, *HIP_FLAGS, *extra_flags, f"-D{define}={n}", "-c", "--save-temps", source, "-o", os.path.join(d, "u.o")]
        subprocess.check_call(cmd, cwd=d, stderr=subprocess.DEVNULL)
        for f in os.listdir(d):
            if f.endswith("gfx950.s"):
                return os.path.join(d, f)
        raise FileNotFoundError("no gfx950 assembly produced")

    with ThreadPoolExecutor(_jobs()) as ex:
        parts = list(ex.map(one, range(units)))
    out = os.path.join(out_dir, name)
    with open(out, "w") as f:
        for part in parts:
            with open(part) as g:
                f.write(g.read())
            f.write("\n")
    return out


def assembly(out_dir: str, extra_flags=()) -> str:
    """Write the gfx950 assembly of every GEMM and convolution kernel to out_dir (one file); returns its path."""
    return _assembly(out_dir, "igc-kernels-gfx950.s", LAUNCH_SOURCE, "IGC_LAUNCH_UNIT", LAUNCH_UNITS, extra_flags)


def ffn_assembly(out_dir: str, extra_flags=()) -> str:
    """The same for the kernels of the feed-forward products."""
    return _assembly(out_dir, "ffn-kernels-gfx950.s", FFN_LAUNCH_SOURCE, "IGC_FFN_UNIT", FFN_LAUNCH_UNITS, extra_flags)


def i8_assembly(out_dir: str, extra_flags=()) -> str:
    """The same for the kernels of the products in 8 bits."""
    return _assembly(out_dir, "i8-kernels-gfx950.s", I8_LAUNCH_SOURCE, "IGC_I8_UNIT", I8_LAUNCH_UNITS, extra_flags)


def rows_assembly(out_dir: str, extra_flags=()) -> str:
    """The same for the row operators."""
    return _assembly(out_dir, "rows-kernels-gfx950.s", ROWS_SOURCE, "IGC_ROWS_UNIT", 1, extra_flags)


if __name__ == "__main__":
    print(build(verbose=True))
    sys.exit(0)
