"""Build libqswiglu.so in-tree with nvcc for sm_103a (GB300), and the C++ binding of
the block operators to torch tensors with g++.

Each translation unit compiles in parallel; the shared libraries land in
``quantized_swiglu_mlp_gb300/lib/``.  No CMake, no torch extension machinery.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "lib")
LIB_PATH = os.path.join(OUT_DIR, "libqswiglu.so")
SOURCES = ["qsw_api.cu", "qsw_gemv.cu", "qsw_gemv_stream.cu", "qsw_prefill.cu", "qsw_elementwise.cu",
           "qsw_block_api.cu", "qsw_fp4.cu", "qsw_fp4_gemm.cu", "qsw_moe.cu", "qsw_norm.cu",
           "qsw_attention_api.cu", "qsw_rope.cu", "qsw_attention.cu", "qsw_attention_tc.cu"]
HEADERS = ["qsw_device.cuh", "qsw_smallm.cuh", "qsw_fp4.cuh", "qsw_tiles.h", "qsw_attention.cuh", "qsw_internal.h",
           "qsw_once.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(verbose_ptxas: bool) -> list[str]:
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
                "-I", os.path.join(ROOT, "include")]
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


# The sources each kernel is compiled from (for kernel_hash).
KERNEL_SOURCES = {
    "gemv_stream": ["qsw_gemv_stream.cu", "qsw_smallm.cuh", "qsw_device.cuh"],
    "gemv": ["qsw_gemv.cu", "qsw_smallm.cuh", "qsw_device.cuh"],
    "prefill": ["qsw_prefill.cu", "qsw_device.cuh"],
}


def _hash(names) -> str:
    import hashlib
    h = hashlib.sha256()
    for name in sorted(names):
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(name.encode())
            h.update(f.read())
    return h.hexdigest()[:12]


def source_hash() -> str:
    """Short hash of every source the library is built from."""
    return _hash(SOURCES + HEADERS)


def kernel_hash(kernel: str) -> str:
    """Short hash of the sources one kernel is compiled from (used to tell
    whether a stored profile still describes that kernel)."""
    return _hash(KERNEL_SOURCES[kernel])


DEBUG_LIB_PATH = os.path.join(OUT_DIR, "libqswiglu_debug.so")
# (library, object folder, extra nvcc flags): the regular build and the debug
# build (device-side address/copy checks and NaN-filled staging, QSW_DEBUG_BOUNDS)
VARIANTS = ((LIB_PATH, "obj", []), (DEBUG_LIB_PATH, "obj_debug", ["-DQSW_DEBUG_BOUNDS"]))


def _stale(lib: str) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    deps.append(os.path.join(ROOT, "include", "qswiglu.h"))
    return any(os.path.getmtime(d) > t for d in deps)


# The binding of the block operators: a CPython module over torch's C++ headers.
NATIVE_SOURCE = os.path.join(CSRC, "qsw_torch.cpp")
NATIVE_PATH = os.path.join(OUT_DIR, "_qsw_torch.so")
NATIVE_STAMP = NATIVE_PATH + ".built_for"


def _native_target() -> str:
    """What the binding is built for: another torch or Python needs another one."""
    return f"torch {importlib.metadata.version('torch')}, {sys.implementation.cache_tag}"


def _native_stale() -> bool:
    if not os.path.exists(NATIVE_PATH) or not os.path.exists(NATIVE_STAMP):
        return True
    with open(NATIVE_STAMP) as f:
        if f.read() != _native_target():
            return True
    t = os.path.getmtime(NATIVE_PATH)
    return any(os.path.getmtime(d) > t for d in (NATIVE_SOURCE, os.path.join(ROOT, "include", "qswiglu.h")))


def _build_native() -> None:
    os.makedirs(OUT_DIR, exist_ok=True)
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = NATIVE_PATH + f".tmp{os.getpid()}"
    include = [os.path.join(ROOT, "include"), os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include"),
               sysconfig.get_path("include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           *(a for d in include for a in ("-isystem", d)), NATIVE_SOURCE, "-o", tmp,
           "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on qsw_torch.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE_PATH)
    with open(NATIVE_STAMP, "w") as f:
        f.write(_native_target())


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile both libraries and the binding (every translation unit at once)
    and return the regular library's path."""
    todo = [v for v in VARIANTS if force or _stale(v[0])]
    native = force or _native_stale()
    if not todo:
        if native:
            _build_native()
        return LIB_PATH
    cc = nvcc()
    flags = _flags(verbose_ptxas)
    for _, objdir, _ in todo:
        os.makedirs(os.path.join(OUT_DIR, objdir), exist_ok=True)

    def compile_one(job) -> str:
        src, objdir, extra = job
        obj = os.path.join(OUT_DIR, objdir, src.replace(".cu", ".o"))
        cmd = [cc, *flags, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose_ptxas:
            sys.stderr.write(r.stderr)
        return obj

    jobs = [(src, objdir, extra) for _, objdir, extra in todo for src in SOURCES]
    with ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        binding = ex.submit(_build_native) if native else None
        objs = list(ex.map(compile_one, jobs))
        if binding:
            binding.result()
    for n, (lib, _, _) in enumerate(todo):
        tmp = lib + f".tmp{os.getpid()}"
        mine = objs[n * len(SOURCES):(n + 1) * len(SOURCES)]
        r = subprocess.run([cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *mine], capture_output=True,
                           text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
