"""Builds libtg.so (the C ABI of include/tg.h) in-tree with nvcc for sm_103a.

    python -m persistent_warp_specialized_gb300._build [--force] [-v]

Five translation units compile in parallel (kernels and C-ABI host code) and are
linked into ``persistent_warp_specialized_gb300/libtg.so`` with the CUDA runtime linked
statically.  Beside them, where torch is installed, ``tg_torch.so``: the CPython module by which
Python calls the products with fused epilogues on torch tensors.  It needs g++, Python's headers and
a torch with CUDA, which the library and all other calls do without: where it cannot be built, the
reason is printed and kept for the first call that needs the module.  Stamps of the sources and flags
(for the module of torch's and Python's versions too) skip rebuilding when nothing changed.
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
TORCH_STAMP = os.path.join(BUILD_DIR, "tg_torch.stamp")
TORCH_ERROR = os.path.join(BUILD_DIR, "tg_torch.error")   # why it could not be built

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


def _hash(paths, *texts):
    """sha256 of files (by path relative to the repository) and texts."""
    h = hashlib.sha256()
    for path in paths:
        h.update(os.path.relpath(path, ROOT).encode())
        with open(path, "rb") as f:
            h.update(f.read())
    for text in texts:
        h.update(text.encode())
    return h.hexdigest()


HEADER = os.path.join(ROOT, "include", "tg.h")


def _stamp():
    """What libtg.so is built from."""
    names = sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh", ".h")))
    return _hash([HEADER] + [os.path.join(CSRC, n) for n in names], " ".join(FLAGS))


def _torch_stamp(root):
    """What tg_torch.so is built from, torch's version file and Python's version among it."""
    try:
        with open(os.path.join(root, "version.py")) as f:
            version = f.read()
    except OSError:
        version = ""
    return _hash([HEADER, os.path.join(CSRC, TORCH_SOURCE)], root, version, sys.version)


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
    # the products with fused epilogues and the kernels around them, profiled together
    "fused_products": ["tg_config.h", "tg_ptx.cuh", "tg_tile_scheduler.cuh", "tg_linear_config.h",
                       "tg_linear_units.h", "tg_linear_kernel.cuh", "tg_few_config.h",
                       "tg_few_kernel.cuh", "tg_gated_kernel.cuh", "tg_outer_kernel.cuh",
                       "tg_xent_kernel.cuh"],
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


def _read(path):
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def _write(path, text):
    with open(path, "w") as f:
        f.write(text)


def torch_error():
    """Why tg_torch.so could not be built the last time, or None."""
    return _read(TORCH_ERROR)


def _start(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    except OSError as e:
        raise RuntimeError(f"{cmd[0]}: {e}") from e


def _finish(proc, what, verbose=False):
    """Waits for a command of _start; raises with its output if it failed."""
    text = proc.communicate()[0].decode(errors="replace")
    if proc.returncode != 0:
        raise RuntimeError(f"{what}\n{text}")
    if verbose:
        print(text, end="", flush=True)


def _gxx():
    return shutil.which("g++") or "g++"


def _start_torch(root, cc, obj, verbose):
    return _start([_gxx(), "-O2", "-std=c++17", "-fPIC", "-Wall",
                   "-I", os.path.join(root, "include"),
                   "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                   "-I", sysconfig.get_paths()["include"],
                   "-I", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include"),
                   "-c", os.path.join(CSRC, TORCH_SOURCE), "-o", obj], verbose)


def _link_torch(root, obj, verbose):
    tmp = TORCH_PATH + ".tmp"
    _finish(_start([_gxx(), "-shared", "-o", tmp, obj, "-L", os.path.join(root, "lib"),
                    "-L", os.path.dirname(LIB_PATH), "-ltorch_python", "-ltorch_cpu", "-lc10",
                    "-lc10_cuda", "-l:libtg.so", "-Wl,-rpath,$ORIGIN"], verbose), "link failed:")
    os.replace(tmp, TORCH_PATH)


def _remove(path):
    if os.path.exists(path):
        os.remove(path)


def build(force=False, verbose=False, ptxas_info=False):
    """Compile libtg.so, and tg_torch.so beside it, if their sources changed; returns libtg.so's path.
    Raises if libtg.so cannot be built (torch_error() says whether tg_torch.so could be)."""
    stamp = _stamp()
    root = _torch_dir()
    torch_stamp = _torch_stamp(root) if root else None
    library = force or not os.path.exists(LIB_PATH) or _read(STAMP) != stamp
    # a failure is kept too: it is tried again when something changed, or by force
    module = root is not None and (
        force or _read(TORCH_STAMP) != torch_stamp
        or not (os.path.exists(TORCH_PATH) or os.path.exists(TORCH_ERROR)))
    if not library and not module:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    torch_obj, torch_proc, why = os.path.join(BUILD_DIR, "tg_torch.o"), None, None
    if module:
        try:
            torch_proc = _start_torch(root, cc, torch_obj, verbose)
        except RuntimeError as e:
            why = str(e)
    if library:
        extra = ["-Xptxas", "-v"] if ptxas_info else []
        objs, procs, failed = [], [], []
        for src in SOURCES:
            obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
            objs.append(obj)
            procs.append((src, _start([cc] + FLAGS + PARALLEL + extra
                                      + ["-c", os.path.join(CSRC, src), "-o", obj], verbose)))
        for src, p in procs:
            try:
                _finish(p, f"--- {src}", verbose or ptxas_info)
            except RuntimeError as e:
                failed.append(str(e))
        if failed:
            if torch_proc is not None:
                torch_proc.communicate()
            raise RuntimeError("nvcc failed:\n" + "\n".join(failed))
        tmp = LIB_PATH + ".tmp"
        _finish(_start([cc] + ARCH + ["-shared", "-Xlinker", "-soname=libtg.so", "-o", tmp] + objs,
                       verbose), "link failed:")
        os.replace(tmp, LIB_PATH)
        _write(STAMP, stamp)
    if module:
        try:
            if torch_proc is not None:
                _finish(torch_proc, f"--- {TORCH_SOURCE}", verbose)
                _link_torch(root, torch_obj, verbose)
        except RuntimeError as e:
            why = str(e)
        if why is None:
            _remove(TORCH_ERROR)
        else:
            _remove(TORCH_PATH)      # not one of other sources
            _write(TORCH_ERROR, why)
            print(f"tg_torch.so was not built, so the fused products cannot be called on torch tensors "
                  f"(--force tries again): {why}", file=sys.stderr)
        _write(TORCH_STAMP, torch_stamp)
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv)
    print(LIB_PATH)
