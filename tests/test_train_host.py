"""The C ABI's host code built with g++ against stand-ins for the CUDA runtime and the kernels (no GPU):
what the weight gradient is set up with and launches."""

import os
import shutil
import subprocess

import pytest

from persistent_warp_specialized_gb300 import _build
from wgrad_shapes import PAIRS, WAYS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not found")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(_build.nvcc())))),
                        "include")
    out = str(tmp_path_factory.mktemp("host") / "train_host_driver")
    # kernels that no test reaches are left undefined
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", cuda, "-I", _build.CSRC, "-x", "c++",
                    os.path.join(ROOT, "tests", "train_host_driver.cpp"),
                    os.path.join(_build.CSRC, "tg_api.cu"),
                    os.path.join(_build.CSRC, "tg_train_api.cu"),
                    "-Wl,--unresolved-symbols=ignore-all", "-o", out], check=True)
    return out


KEYS = ("rc", "halves", "splits", "blocks_per_split", "k_blocks", "split_from", "units", "grid",
        "tma_scales", "workspace", "setups")


def run(driver, rows, cols, outs, gemm_pairs=76, wgrad_pairs=76, scale_offset=0):
    """(the GEMM's rc and workers, set-ups before the weight gradient's call, what that launches)"""
    args = (gemm_pairs, wgrad_pairs, rows, cols, outs, scale_offset)
    text = subprocess.run([driver] + [str(a) for a in args], check=True, capture_output=True,
                          text=True).stdout.split("\n")
    gemm, setup, wgrad = (tuple(int(v) for v in line.split()[1:]) for line in text[:3])
    return gemm, setup[0], dict(zip(KEYS, wgrad))


def test_the_gemm_does_not_wait_for_the_weight_gradient(driver):
    gemm, before, wgrad = run(driver, 8192, 8192, 8192)
    assert gemm == (0, 76) and before == 0          # nothing of it is set up for a GEMM
    assert wgrad["rc"] == 0 and wgrad["grid"] == 152 and wgrad["setups"] == 1   # once, two calls


@pytest.mark.parametrize("gemm_pairs,wgrad_pairs", [(76, 40), (40, 76)])
def test_each_has_its_own_resident_pairs(driver, gemm_pairs, wgrad_pairs):
    gemm, _, wgrad = run(driver, 8192, 8192, 8192, gemm_pairs, wgrad_pairs)
    assert gemm == (0, gemm_pairs)
    assert wgrad["rc"] == 0 and wgrad["grid"] == 2 * wgrad_pairs


@pytest.mark.parametrize("wgrad_pairs", [-1, 0])
def test_without_the_weight_gradient_the_gemm_still_runs(driver, wgrad_pairs):
    gemm, _, wgrad = run(driver, 512, 512, 512, wgrad_pairs=wgrad_pairs)
    assert gemm == (0, 76)
    assert wgrad["rc"] == -3 and wgrad["halves"] == 0    # TG_ERR_CUDA, and no launch


@pytest.mark.parametrize("shape", WAYS)
def test_what_is_launched(driver, shape):
    halves, splits, half_units, most, tma = WAYS[shape]
    _, _, w = run(driver, *shape)
    assert w["rc"] == 0 and (w["halves"], w["splits"]) == (halves, splits)
    assert w["units"] - w["split_from"] == half_units
    assert -(-w["units"] * w["splits"] // (w["grid"] // 2)) == most
    assert bool(w["tma_scales"]) == tma
    # scales off the 16-byte grid are copied word by word
    assert run(driver, *shape, scale_offset=4)[2]["tma_scales"] == 0


def test_ranges_cover_the_tokens(driver):
    for rows in (9000, 10369, 16000, 20000, 30000, 65536):
        for cols, outs in ((40, 16), (512, 1024), (2000, 1000), (300, 520)):
            _, _, w = run(driver, rows, cols, outs)
            assert w["k_blocks"] == -(-rows // 64)
            assert (w["splits"] - 1) * w["blocks_per_split"] < w["k_blocks"]
            assert w["splits"] * w["blocks_per_split"] >= w["k_blocks"]
            assert w["units"] * w["splits"] <= PAIRS or w["splits"] == 1
