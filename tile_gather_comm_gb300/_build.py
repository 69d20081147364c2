"""Build libtgc.so in-tree with nvcc for sm_103a (no torch extension machinery), and _ops.so, the
native argument marshalling, with g++ against Python's and torch's headers.

Each translation unit under csrc/ is compiled in parallel to an object file,
then nvcc links them into ``tile_gather_comm_gb300/libtgc.so`` with the CUDA
runtime linked statically.  Host code is plain C++17 (no architecture-specific
intrinsics), so the same command builds on x86_64 and aarch64.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libtgc.so")
OPS = os.path.join(PKG, "_ops.so")
OPS_STAMP = os.path.join(PKG, "_build", "ops.stamp")  # the Python and torch that _ops.so was built against
SOURCES = ["api.cu", "tgather.cu", "gemm.cu", "noalloc.cu", "ipc.cu", "linear.cu", "linear_gemm.cu", "linear_split.cu", "block_norm.cu",
           "rope.cu", "paged_attention.cu", "kv_pages.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found (CUDA toolkit required to build libtgc.so)")
    return cand


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "tgc.h"))
    files.append(os.path.abspath(__file__))
    return files


def _newer_than_inputs(path: str) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in _inputs())


def _ops_needs() -> str:
    import torch
    return f"Python {sys.version}\ntorch {torch.__version__}\n"


def _ops_up_to_date() -> bool:
    """Newer than its sources, and built against this Python and this torch: another's ABI may differ."""
    if not _newer_than_inputs(OPS) or not os.path.exists(OPS_STAMP):
        return False
    with open(OPS_STAMP, encoding="utf-8") as f:
        return f.read() == _ops_needs()


def up_to_date() -> bool:
    return _newer_than_inputs(LIB) and _ops_up_to_date()


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    with concurrent.futures.ThreadPoolExecutor(1) as ex:
        ops = ex.submit(_compile_ops) if force or not _ops_up_to_date() else None
        if force or not _newer_than_inputs(LIB):
            _compile(os.path.join(PKG, "_build"), LIB, [], verbose, ptxas_info)
        if ops is not None:
            ops.result()
    return LIB


def _compile_ops() -> None:
    """_ops.so: host code only, against the headers of the Python and torch that run this."""
    import sysconfig

    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = OPS + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), os.path.join(CSRC, "binding.cpp"), "-o", tmp,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OPS)
    os.makedirs(os.path.dirname(OPS_STAMP), exist_ok=True)
    with open(OPS_STAMP, "w", encoding="utf-8") as f:
        f.write(_ops_needs())


def build_variant(out_dir: str, defines: dict, sources: list | None = None) -> str:
    """Build the library with compile-time settings changed (e.g. {"TGC_COPY_LSU": 0})
    into out_dir/libtgc.so and return its path; the in-tree library is not touched.
    ``sources``: the only files that the settings concern; the others' objects are the in-tree build's."""
    flags = [f"-D{k}={v}" for k, v in sorted(defines.items())]
    return _compile(out_dir, os.path.join(out_dir, "libtgc.so"), flags, False, False, sources or SOURCES)


def _compile(out_dir: str, lib_path: str, extra: list, verbose: bool, ptxas_info: bool, sources=SOURCES) -> str:
    os.makedirs(out_dir, exist_ok=True)
    common = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-Wall", "-I", INCLUDE, "-I", CSRC, *extra]
    if ptxas_info:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(out_dir, os.path.splitext(src)[0] + ".o")
        cmd = common + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    kept = [os.path.join(PKG, "_build", os.path.splitext(s)[0] + ".o") for s in SOURCES if s not in sources]
    with concurrent.futures.ThreadPoolExecutor(len(sources)) as ex:
        objs = list(ex.map(compile_one, sources)) + kept
    tmp = lib_path + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
