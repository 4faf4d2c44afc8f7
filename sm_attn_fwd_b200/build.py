"""Ahead-of-time build of the CUDA library for sm_100a (B200).

Compiles ``csrc/*.cu`` with nvcc into ``_lib/libattn_b200.so`` inside the
package directory (no JIT cache, nothing installed elsewhere), and
``csrc/torch_binding.cpp``, the native part of the Python binding, into
``_lib/attn_torch.so`` beside it.  Run as
``python -m sm_attn_fwd_b200.build`` or call :func:`build`.
"""
from __future__ import annotations

import hashlib
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libattn_b200.so")
EXT = os.path.join(LIBDIR, "attn_torch.so")
EXT_SOURCE = "torch_binding.cpp"
EXT_MARK = b"attn_torch built for "  # in the object, before its stamp
SOURCES = ["attn_api.cu", "attn_kernels.cu", "attn_prefill.cu", "attn_short.cu", "attn_noalloc.cu",
           "attn_backward.cu", "attn_cache_q8.cu", "attn_decode_rows.cu",
           "attn_decode_q8_wide.cu", "attn_prefix.cu"]
HEADERS = ["attn_params.h", "attn_bwd_params.h", "ptx.cuh", "host_once.h", "prefill_common.cuh",
           "softmax_row.cuh", "cache_q8.cuh", "decode_params.h",
           "attn_prefix_params.h", "decode_sched.cuh"]

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC,-O2,-Wall",
    "-Xptxas", "-v",
    "--expt-relaxed-constexpr",
]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def source_digest(files=("attn_prefill.cu", "prefill_common.cuh", "ptx.cuh", "attn_params.h",
                         "softmax_row.cuh")) -> str:
    """Digest of one kernel's sources and the flags (identifies a profiled
    build); by default the prefill kernel's."""
    h = hashlib.sha256()
    for name in files:
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(f.read())
    h.update(" ".join(NVCC_FLAGS).encode())
    return h.hexdigest()[:16]


def _digest() -> str:
    h = hashlib.sha256()
    for name in SOURCES + HEADERS:
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(f.read())
    with open(os.path.join(ROOT, "include", "attn.h"), "rb") as f:
        h.update(f.read())
    h.update(" ".join(NVCC_FLAGS).encode())
    return h.hexdigest()[:16]


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if its sources changed; return the .so path."""
    os.makedirs(LIBDIR, exist_ok=True)
    stamp = os.path.join(LIBDIR, "libattn_b200.sha")
    digest = _digest()
    if not force and lib_is_current():
        return LIB
    nvcc = nvcc_path()
    objs = []
    for src in SOURCES:
        obj = os.path.join(LIBDIR, src.replace(".cu", ".o"))
        cmd = [nvcc, *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c",
               os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stdout + r.stderr)
        objs.append(obj)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", tmp, *objs,
           "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    for obj in objs:
        os.remove(obj)
    with open(stamp, "w") as f:
        f.write(digest)
    return LIB


EXT_INPUTS = (os.path.join(CSRC, EXT_SOURCE), os.path.join(ROOT, "include", "attn.h"))


def _ext_mark(parts: int = 2) -> bytes:
    """What the native part of the binding is built for: this interpreter and torch (it uses
    torch's C++ interface), then its source and the C ABI it calls."""
    import torch

    env = hashlib.sha256(f"{sys.version} {torch.__version__}".encode()).hexdigest()[:16]
    if parts == 1:
        return EXT_MARK + env.encode()
    h = hashlib.sha256()
    for path in EXT_INPUTS:
        with open(path, "rb") as f:
            h.update(f.read())
    return EXT_MARK + f"{env} {h.hexdigest()[:16]}".encode()


def is_current(ext: str = EXT) -> bool:
    """Whether the native part of the binding was built for this interpreter and torch and,
    where its sources are there to compare, from them (the object says so itself): another
    build's must not be loaded."""
    parts = 2 if all(os.path.exists(path) for path in EXT_INPUTS) else 1
    with open(ext, "rb") as f:
        return _ext_mark(parts) in f.read()


def lib_is_current() -> bool:
    """Whether the library was built from these sources."""
    stamp = os.path.join(LIBDIR, "libattn_b200.sha")
    if not os.path.exists(LIB) or not os.path.exists(stamp):
        return False
    with open(stamp) as f:
        return f.read().strip() == _digest()


def build_ext(force: bool = False, verbose: bool = False) -> str:
    """Compile the native part of the binding if its sources, the interpreter or torch
    changed; return its path."""
    import sysconfig

    import torch

    lib = build(force, verbose)
    if not force and os.path.exists(EXT) and is_current(EXT):
        return EXT
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    includes = [os.path.join(t, "include"), os.path.join(cuda, "include"),
                sysconfig.get_paths()["include"]]
    tmp = EXT + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f'-DATTN_TORCH_MARK="{_ext_mark().decode()}"',
           "-I", os.path.join(ROOT, "include")]
    for path in includes:
        cmd += ["-isystem", path]
    cmd += [os.path.join(CSRC, EXT_SOURCE), "-o", tmp, "-L" + os.path.dirname(lib),
            "-l:" + os.path.basename(lib), "-Wl,-rpath,$ORIGIN",
            "-L" + os.path.join(t, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch",
            "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {EXT_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)
    return EXT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
    print(build_ext(force="--force" in sys.argv))
