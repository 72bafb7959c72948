"""Build the CUDA library (libattn.so, sm_103a) in-tree with nvcc.

    python -m transformer_scaled_dot_fwd_gb300.build [--force] [--verbose-ptxas]

Each .cu file compiles to an object in parallel; the objects link into
``transformer_scaled_dot_fwd_gb300/libattn.so`` with the CUDA runtime linked
statically.  The driver API is reached through cudaGetDriverEntryPointByVersion,
so no link against libcuda is needed.  csrc/binding.cpp, the Python binding of the
serving entry points, compiles beside them with the host compiler against the
installed torch, whose version its file name carries.  Where it cannot be compiled
(no Python headers, another torch's C++ headers) the library is built all the same,
with a warning, and the entry points take their checked path in Python.
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libattn.so")
SOURCES = ["api.cu", "prefill_tc.cu", "prefill_f32.cu", "decode.cu", "decode_gqa.cu", "decode_tc.cu", "decode_f32.cu", "decode_noalloc.cu", "debug.cu",
           "rope.cu", "tile_f32.cu", "tree_tc.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found")
    return exe


def binding_path(version: str) -> str:
    """The binding built for torch ``version``."""
    return os.path.join(PKG, f"_binding.torch{version}.so")


def _binding_command():
    """(output, command) of the binding for the installed torch; None without torch."""
    try:
        import torch
    except ImportError:
        return None
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    out = binding_path(torch.__version__)
    return out, [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
                 f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
                 "-isystem", os.path.join(root, "include"),
                 "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                 "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
                 os.path.join(CSRC, "binding.cpp"), "-o", out + f".tmp{os.getpid()}",
                 "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def _newest_input_mtime():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def build(force: bool = False, verbose_ptxas: bool = False, quiet: bool = False) -> str:
    """Compile every kernel file for sm_103a, link libattn.so and compile the binding;
    returns the library's path.  A binding that does not compile is a warning."""
    newest = _newest_input_mtime()

    def stale(path):
        return force or not os.path.exists(path) or os.path.getmtime(path) < newest

    binding = _binding_command()
    started = None
    if binding and stale(binding[0]):
        started = subprocess.Popen(binding[1], stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    try:
        if stale(LIB_PATH):
            _build_library(verbose_ptxas, quiet)
    finally:
        if started:
            text = started.communicate()[0].decode(errors="replace")
    if started and started.returncode == 0:
        os.replace(binding[1][binding[1].index("-o") + 1], binding[0])
    elif started:
        if os.path.exists(binding[0]):
            os.remove(binding[0])  # of older sources: its calls may not be the library's any more
        warnings.warn(f"{os.path.basename(binding[1][0])} could not compile csrc/binding.cpp; the serving entry points "
                      f"take their checked path in Python, some 10 us more a call:\n{text}", RuntimeWarning)
    return LIB_PATH


def _build_library(verbose_ptxas: bool, quiet: bool) -> None:
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    flags = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
                    "-I", INCLUDE, "-I", CSRC]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]
    procs, objs = [], []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [nvcc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((src, text))
        elif text.strip() and (verbose_ptxas or not quiet):
            sys.stderr.write(f"--- {src}\n{text}")
    if failed:
        msg = "\n".join(f"--- {s}\n{t}" for s, t in failed)
        raise RuntimeError(f"nvcc failed:\n{msg}")
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    link = [nvcc] + ARCH + ["-shared", "-Xcompiler", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, LIB_PATH)


def main():
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose_ptxas=args.verbose_ptxas))


if __name__ == "__main__":
    main()
