"""Build libwtconv.so (the C-ABI WTConv library) in-tree with nvcc for sm_103a, and _binding.so, the
compiled Python binding of the operators beside the layer, with g++ against the installed PyTorch.

Each translation unit is compiled in parallel; the library is relinked only when a source or
header is newer than it.  The results land next to this file, so they are found without any
installation step.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
CSRC_TRAIN = os.path.join(CSRC, "train")  # operators beside the layer: gated scan, AdamW, gradient norm
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libwtconv.so")
CSRC_BINDING = os.path.join(CSRC, "binding")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_KEY = os.path.join(PKG, "_binding.key")  # the PyTorch and Python that _binding.so was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu"))) + sorted(glob.glob(os.path.join(CSRC_TRAIN, "*.cu")))


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile_binding() -> list[tuple[list[str], str]]:
    """Commands that compile the binding's objects, each with its object."""
    import torch

    torch_dir = os.path.dirname(torch.__file__)
    includes = [INCLUDE, os.path.join(torch_dir, "include"),
                os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", *["-I" + d for d in includes],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    objs = [(src, os.path.join(BUILD, "binding_" + os.path.basename(src)[:-4] + ".o"))
            for src in sorted(glob.glob(os.path.join(CSRC_BINDING, "*.cpp")))]
    return [([*cmd, "-c", src, "-o", obj], obj) for src, obj in objs]


def _binding_key() -> str:
    import torch

    return f"torch {torch.__version__} at {os.path.dirname(torch.__file__)}, C++11 ABI {torch._C._GLIBCXX_USE_CXX11_ABI}, " \
        f"Python {sysconfig.get_config_var('SOABI')}\n"


def binding_stale() -> bool:
    """Whether the binding is missing, older than its sources, or built for another PyTorch or Python."""
    if _stale(BINDING, [*glob.glob(os.path.join(CSRC_BINDING, "*")), *glob.glob(os.path.join(INCLUDE, "*.h")), __file__]):
        return True
    try:
        with open(BINDING_KEY) as f:
            return f.read() != _binding_key()
    except FileNotFoundError:
        return True


def _link_binding(objs: list[str]) -> None:
    import torch

    lib_dir = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".{os.getpid()}.tmp"
    subprocess.run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, *objs, "-L" + os.path.dirname(LIB), "-l:libwtconv.so",
                    "-Wl,-rpath,$ORIGIN", "-L" + lib_dir, "-Wl,-rpath," + lib_dir, "-ltorch_python", "-ltorch", "-ltorch_cpu",
                    "-ltorch_cuda", "-lc10", "-lc10_cuda"], check=True)
    os.replace(tmp, BINDING)
    with open(BINDING_KEY + f".{os.getpid()}.tmp", "w") as f:
        f.write(_binding_key())
    os.replace(f.name, BINDING_KEY)


def _start(cmd: list[str], verbose: bool):
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    return cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _finish(procs) -> None:
    failed = []
    for cmd, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((cmd, out.decode(errors="replace")))
    if failed:
        msg = "\n".join(" ".join(c) + "\n" + o for c, o in failed)
        raise RuntimeError("compilation failed:\n" + msg)


def _build_library(force: bool, verbose: bool) -> None:
    srcs = sources()
    headers = [h for d in (CSRC, CSRC_TRAIN, INCLUDE) for pat in ("*.h", "*.cuh")
               for h in glob.glob(os.path.join(d, pat))]
    if not force and not _stale(LIB, srcs + headers + [__file__]):
        return
    procs = []
    objs = []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        # a layer kernel uses the layer's headers, an operator of csrc/train that folder's own
        used = [h for h in headers if os.path.dirname(h) in (INCLUDE, os.path.dirname(src))]
        if not force and not _stale(obj, [src, *used, __file__]):
            continue
        procs.append(_start([nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj], verbose))
    _finish(procs)
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "shared", "-Xlinker", "-soname=libwtconv.so", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False, binding: bool = True) -> str:
    """Build what is missing or stale: the library, and with ``binding`` the compiled binding beside it;
    returns the library's path.  The library needs nothing of the binding, and is built where that fails."""
    os.makedirs(BUILD, exist_ok=True)
    compiling, failure, objs = [], None, []
    if binding and (force or binding_stale()):
        try:
            for cmd, obj in _compile_binding():
                compiling.append(_start(cmd, verbose))
                objs.append(obj)
        except OSError as e:  # no compiler for it
            failure = e
    try:
        _build_library(force, verbose)
    except BaseException:
        for _, p in compiling:
            p.communicate()
        raise
    if failure is not None:
        raise failure
    if compiling:
        _finish(compiling)
        _link_binding(objs)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
