"""Build libawqsearch.so in-tree with nvcc for sm_100a (B200).

    python -m post_quantization_column_b200.build [--force] [--verbose]

and _decode.so, the CPython binding of the decode-step operators, with the C++ compiler where
torch and Python's headers are there (programs that use the C library alone need neither).

Objects go to ``post_quantization_column_b200/_build/`` (not committed); the shared
library is written next to this file so the package finds it without installation.
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libawqsearch.so")
BINDING = os.path.join(PKG, "_decode.so")
BINDING_KEY = os.path.join(BUILD, "_decode.key")
SOURCES = ["awq_api.cu", "k_statistic.cu", "k_qdq.cu", "k_loss_gemm.cu", "k_clip.cu", "k_w4a16.cu", "k_module.cu", "k_attn.cu", "awq_noalloc.cu", "gemm_policy.cu",
           "awq_decode.cu", "k_rmsnorm.cu", "k_rmsnorm_odd.cu", "k_kv_append.cu", "k_paged_attn.cu"]
HEADERS = ["awq_device.cuh", "awq_kernels.h", "qdq_tile.cuh", "decode_kernels.h", "decode_entry.h", "rmsnorm.cuh"]

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
# IEEE division, square root and denormals everywhere: the QDQ must match the
# oracle bit for bit, so no fast-math and no flush-to-zero.
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "-prec-div=true", "-prec-sqrt=true", "-ftz=false", "-fmad=true",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libawqsearch.so")
    return path


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "awq_search.h")]
    objs, cmds = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            cmd = [nvcc(), *ARCH, *FLAGS, "-c", s, "-o", o]
            if ptxas_verbose:
                cmd += ["-Xptxas", "-v"]
            if verbose:
                print(" ".join(cmd), flush=True)
            cmds.append(cmd)
    # the translation units are independent: compile them side by side
    from concurrent.futures import ThreadPoolExecutor
    with ThreadPoolExecutor(max_workers=max(1, min(len(cmds), os.cpu_count() or 1))) as pool:
        for r in pool.map(lambda c: subprocess.run(c, capture_output=not verbose and not ptxas_verbose, text=True),
                          cmds):
            if r.returncode != 0:
                if r.stdout or r.stderr:
                    sys.stderr.write((r.stdout or "") + (r.stderr or ""))
                raise subprocess.CalledProcessError(r.returncode, r.args)
    if force or _stale(LIB, objs):
        cmd = [nvcc(), *ARCH, "-shared", "-o", LIB, *objs, "-cudart", "static"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    lacking = _binding_lacks()
    if lacking:
        print(f"_decode.so is not built: {lacking}; libawqsearch.so does not need it", file=sys.stderr)
    else:
        build_binding(force, verbose)
    return LIB


def _binding_lacks() -> str | None:
    """What building _decode.so lacks here, None if nothing."""
    import sysconfig
    try:
        import torch
    except ImportError as e:
        return f"torch does not import ({e})"
    if torch.version.cuda is None:
        return "torch is built without CUDA"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers are not installed"
    if not (shutil.which("g++") or shutil.which("c++")):
        return "no C++ compiler found"
    return None


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/decode_binding.cpp against torch's headers and link it to the library next to it."""
    import sysconfig

    import torch
    src = os.path.join(CSRC, "decode_binding.cpp")
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("no C++ compiler found; it is required to build _decode.so")
    t = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", src, "-o", BINDING, f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", os.path.join(t, "include"), "-I", os.path.join(t, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
           "-L", PKG, "-lawqsearch", "-L", os.path.join(t, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
           "-Wl,-rpath,$ORIGIN"]
    # what it was built for: another torch or Python needs another build
    key = "\n".join([torch.__version__, sys.version, *cmd])
    if os.path.exists(BINDING_KEY):
        with open(BINDING_KEY) as f:
            force = force or f.read() != key
    else:
        force = True
    if not (force or _stale(BINDING, [src, os.path.join(CSRC, "decode_entry.h"), os.path.join(ROOT, "include", "awq_search.h")])):
        return BINDING
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.makedirs(BUILD, exist_ok=True)
    with open(BINDING_KEY, "w") as f:
        f.write(key)
    return BINDING


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true", help="print registers / spills / smem per kernel")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose, ptxas_verbose=a.ptxas_verbose))
    return 0


if __name__ == "__main__":
    sys.exit(main())
