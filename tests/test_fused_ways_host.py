"""The sizes of tests/test_fused_exact_gpu.py take every way through the fused products: their host code is built
with g++ against stand-ins for the CUDA runtime and the kernels (no GPU) and says what it launches for each.

Ways of the pair kernel: kk, kn, mn is how A and B lie (k contiguous, or not); -split: K in ranges; -segments:
more than one accumulator's sums; -two: two products in the launch; -two-along-k, -n: two matrices in an
operand's place; -added: sums over pieces of a vocabulary (-fewer: in fewer ranges than the first piece's).
"""

import os
import shutil
import subprocess

import pytest

from fused_exact_sizes import GATED_BWD, GATED_FWD, INPUT_GRADS, XENT_BWD, XENT_FWD
from persistent_warp_specialized_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not found")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(_build.nvcc())))),
                        "include")
    out = str(tmp_path_factory.mktemp("host") / "fused_ways_driver")
    # kernels that no test reaches are left undefined
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", cuda, "-I", _build.CSRC, "-x", "c++",
                    os.path.join(ROOT, "tests", "fused_ways_driver.cpp"),
                    os.path.join(_build.CSRC, "tg_api.cu"),
                    os.path.join(_build.CSRC, "tg_linear_api.cu"),
                    "-Wl,--unresolved-symbols=ignore-all", "-o", out], check=True)
    return out


def few(epi, lies, rows=(16, 32, 64), ranks=(), also=()):
    way = f"few-{epi}-{lies}"
    return {f"{way}-rows{n}" for n in rows} | {f"{way}-ranks{n}" for n in ranks} | {f"{way}-{a}" for a in also}


def pair(epi, lies, *also):
    return {f"pair-{epi}-{lies}"} | {f"pair-{epi}-{lies}-{a}" for a in also}


WAYS = {
    "input_grad": (INPUT_GRADS, few("store", "kk", ranks=(1, 2, 4, 8), also=["groups"])
                   | pair("store", "kk", "split", "segments", "half-units") | {"join1"}),
    "gated_fwd": (GATED_FWD, few("gated", "kn", ranks=(1, 2, 4, 8)) | pair("gated", "kn", "segments", "half-units")
                  | pair("store", "kn", "split", "two-along-n") | {"gated-join"}),
    "gated_bwd": (GATED_BWD, few("store", "kk", ranks=(4, 8), also=["groups", "terms", "two-along-k"])
                  | pair("store", "kk", "two", "two-along-k", "split", "segments", "half-units")
                  | pair("store", "mn", "two", "two-along-n", "split", "segments", "half-units")
                  | {"outer2", "join1", "join2"}),
    "xent_fwd": (XENT_FWD, few("stats", "kk", ranks=(1, 2, 4, 8)) | pair("stats", "kk", "segments", "half-units")
                 | pair("store", "kk", "split") | {"xent-join", "xent-rows"}),
    "xent_bwd": (XENT_BWD, few("dlogits", "kk", ranks=(1, 8)) | few("store", "kn", ranks=(8,), also=["groups", "terms"])
                 | pair("dlogits", "kk", "half-units") | pair("store", "kk", "split")
                 | pair("store", "kn", "two", "split", "segments", "added", "added-split", "added-fewer")
                 | pair("store", "mn", "two", "split", "segments", "half-units")
                 | {"outer1", "join1", "xent-dlogits"}),
}


@pytest.mark.parametrize("operator", WAYS)
def test_every_way_is_taken(driver, operator):
    sizes, ways = WAYS[operator]
    calls = "\n".join(" ".join(map(str, (operator,) + s)) for s in sizes)
    done = subprocess.run([driver], input=calls, capture_output=True, text=True)
    assert done.returncode == 0, done.stdout[-200:]
    lines = done.stdout.splitlines()
    assert len(lines) == len(sizes)
    left = ways - {w for line in lines for w in line.split()}
    assert not left, sorted(left)
