"""Builds liblinattn.so in-tree with nvcc for sm_103a (translation units compiled in parallel), and where torch is
installed, with the C++ compiler, the module that takes ordinary calls from its tensors to the library (csrc/bind.cpp).

Usage: ``python -m chunked_state_scan_causal_gb300.build [--verbose]``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "liblinattn.so")
SOURCES = ["api.cu", "simt.cu", "scan.cu", "tc.cu", "diag.cu", "decode.cu", "gate.cu", "softmax.cu", "gate_vec.cu",
           "pad.cu", "delta.cu", "delta_tc.cu", "paged.cu", "paged8.cu", "rope.cu"]
BIND = "bind.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build liblinattn")


def bind_path() -> str:
    """The module built for the installed torch and Python."""
    import torch
    name = f"_bind_{torch.__version__}_{sys.version_info[0]}{sys.version_info[1]}"
    return os.path.join(OUT_DIR, "".join(c if c.isalnum() or c == "_" else "_" for c in name) + ".so")


def _bind_flags():
    import sysconfig

    import torch
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    include = [sysconfig.get_paths()["include"], os.path.join(cuda, "include"), root,
               os.path.join(root, "torch", "csrc", "api", "include")]
    return ["-std=c++17", "-O2", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-I{d}" for d in include)]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    deps = [*(os.path.join(CSRC, f) for f in deps), os.path.join(HERE, "..", "include", "linattn.h"), os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def _run(cmd, what: str, verbose: bool = False) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(f"--- {what}\n{r.stdout}{r.stderr}")


def _link(out: str, cmd) -> None:
    tmp = out + f".tmp{os.getpid()}"
    _run([*cmd, "-shared", "-o", tmp], "link")
    os.replace(tmp, out)


def _object(src: str) -> str:
    return os.path.join(OUT_DIR, "obj", os.path.splitext(src)[0] + ".o")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA translation unit and link liblinattn.so; returns its path.  The module of the compiled marshalling
    comes with it where torch, its headers and a C++ compiler are; without it calls take the Python way."""
    why = None  # the module is left out
    try:
        module = bind_path()
    except ImportError as e:
        module, why = None, e
    need_lib = force or _stale(LIB, [f for f in os.listdir(CSRC) if f != BIND])
    need_module = module and (force or _stale(module, [BIND]))
    os.makedirs(os.path.join(OUT_DIR, "obj"), exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose else []
    cxx = shutil.which("g++") or "c++"

    def compile_one(src: str) -> None:
        _run([_nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", _object(src)], src, verbose)

    def compile_module() -> None:
        _run([cxx, *_bind_flags(), "-c", os.path.join(CSRC, BIND), "-o", _object(BIND)], BIND, verbose)

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        waiting = ex.submit(compile_module) if need_module else None
        if need_lib:
            list(ex.map(compile_one, SOURCES))
            _link(LIB, [_nvcc(), *ARCH, *map(_object, SOURCES)])
        if waiting:
            import torch
            torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
            try:
                waiting.result()
                _link(module, [cxx, _object(BIND), f"-L{OUT_DIR}", "-llinattn", f"-L{torch_lib}", "-ltorch_python",
                               "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"])
            except (RuntimeError, OSError) as e:
                why = e
    if why:
        sys.stderr.write(f"the compiled marshalling is left out (calls take the Python way): {why}\n")
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv))
