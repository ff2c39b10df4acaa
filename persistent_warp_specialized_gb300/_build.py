"""Builds libtg.so (the C ABI of include/tg.h) in-tree with nvcc for sm_103a.

    python -m persistent_warp_specialized_gb300._build [--force] [-v]

Five translation units compile in parallel (kernels and C-ABI host code) and are
linked into ``persistent_warp_specialized_gb300/libtg.so`` with the CUDA runtime linked
statically.  Beside them, where torch is installed, ``tg_torch.so``: the CPython module by which
Python calls the products with fused epilogues on torch tensors.  A stamp of the sources and flags
(and of torch's and Python's versions) skips rebuilding when nothing changed.
"""

import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libtg.so")
STAMP = os.path.join(BUILD_DIR, "libtg.stamp")
TORCH_SOURCE = "tg_torch.cpp"
TORCH_PATH = os.path.join(HERE, "tg_torch.so")

SOURCES = ["tg_gemm.cu", "tg_train.cu", "tg_api.cu", "tg_train_api.cu", "tg_linear_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                "-Xcompiler", "-Wall", "-diag-suppress", "177"]
# a translation unit's kernels are compiled side by side (tg_gemm.cu: 17 s instead of 75)
PARALLEL = ["-split-compile=0"]


def nvcc():
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand) and not shutil.which(cand):
        raise RuntimeError("nvcc not found; set NVCC or put the CUDA toolkit on PATH")
    return cand


def _torch_dir():
    """Where torch is installed (found without importing it), or None."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def _torch_version(root):
    """What tg_torch.so has to be built again for: torch's version file and Python's version."""
    with open(os.path.join(root, "version.py")) as f:
        return f.read() + sys.version


def _inputs():
    files = [os.path.join(ROOT, "include", "tg.h")]
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h", ".cpp")):
            files.append(os.path.join(CSRC, name))
    return files


def _stamp():
    """sha256 of the library's sources (by path relative to the repository), flags and torch's
    version."""
    h = hashlib.sha256()
    for path in _inputs():
        h.update(os.path.relpath(path, ROOT).encode())
        with open(path, "rb") as f:
            h.update(f.read())
    h.update(" ".join(FLAGS).encode())
    root = _torch_dir()
    h.update(_torch_version(root).encode() if root else b"no torch")
    return h.hexdigest()


# The sources each GEMM kernel's device code is built from (a profile taken of a kernel stays
# valid while these and the flags are unchanged).
KERNEL_SOURCES = {
    "gemm_persistent_ws": ["tg_config.h", "tg_ptx.cuh", "tg_tile_scheduler.cuh",
                           "tg_gemm_kernel.cuh"],
    "gemm_pair_ws": ["tg_config.h", "tg_ptx.cuh", "tg_tile_scheduler.cuh", "tg_gemm_kernel.cuh",
                     "tg_gemm_pair_kernel.cuh"],
    "gemm_pair_wide_ws": ["tg_config.h", "tg_ptx.cuh", "tg_tile_scheduler.cuh", "tg_gemm_kernel.cuh",
                          "tg_gemm_pair_kernel.cuh", "tg_wide_config.h",
                          "tg_gemm_pair_wide_kernel.cuh"],
    "gemm_mxfp8_ws": ["tg_config.h", "tg_ptx.cuh", "tg_tile_scheduler.cuh", "tg_gemm_kernel.cuh",
                      "tg_mx_kernel.cuh"],
    "gemm_mxfp8_pair_ws": ["tg_config.h", "tg_ptx.cuh", "tg_tile_scheduler.cuh",
                           "tg_gemm_kernel.cuh", "tg_gemm_pair_kernel.cuh", "tg_mx_kernel.cuh",
                           "tg_mx_pair_kernel.cuh"],
}


def kernel_stamp(kernel):
    """sha256 of one kernel's device sources and the flags."""
    h = hashlib.sha256()
    for name in KERNEL_SOURCES[kernel]:
        h.update(name.encode())
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(f.read())
    h.update(" ".join(FLAGS).encode())
    return h.hexdigest()


def build(force=False, verbose=False, ptxas_info=False):
    """Compile libtg.so if its sources changed; returns its path."""
    stamp = _stamp()
    root = _torch_dir()
    if (not force and os.path.exists(LIB_PATH) and os.path.exists(STAMP)
            and (root is None or os.path.exists(TORCH_PATH))):
        with open(STAMP) as f:
            if f.read().strip() == stamp:
                return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [cc] + FLAGS + PARALLEL + extra + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    if root is not None:
        obj = os.path.join(BUILD_DIR, "tg_torch.o")
        cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-Wall",
               "-I", os.path.join(root, "include"),
               "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
               "-I", sysconfig.get_paths()["include"],
               "-I", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include"),
               "-c", os.path.join(CSRC, TORCH_SOURCE), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((TORCH_SOURCE,
                      subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append(f"--- {src}\n{text}")
        elif verbose or ptxas_info:
            print(text, end="", flush=True)
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(failed))
    tmp = LIB_PATH + ".tmp"
    cmd = [cc] + ARCH + ["-shared", "-Xlinker", "-soname=libtg.so", "-o", tmp] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, LIB_PATH)
    if root is not None:
        tmp = TORCH_PATH + ".tmp"
        cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp,
               os.path.join(BUILD_DIR, "tg_torch.o"), "-L", os.path.join(root, "lib"), "-L", HERE,
               "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-l:libtg.so",
               "-Wl,-rpath,$ORIGIN"]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
        os.replace(tmp, TORCH_PATH)
    with open(STAMP, "w") as f:
        f.write(stamp)
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv)
    print(LIB_PATH)
