"""The walk over the fused products' units (tg_linear_units.h, the kernel's own) built for the host with g++: in
random launches every tile's every k-block is taken once (no GPU)."""

import os
import shutil
import subprocess

import pytest

from persistent_warp_specialized_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not found")
    out = str(tmp_path_factory.mktemp("units") / "linear_units_driver")
    subprocess.run([cxx, "-O2", "-std=c++17", "-D__host__=", "-D__device__=", "-I", _build.CSRC,
                    os.path.join(ROOT, "tests", "linear_units_driver.cpp"), "-o", out], check=True)
    return out


@pytest.mark.parametrize("seed", range(3))
def test_every_unit_is_taken_once(driver, seed):
    text = subprocess.run([driver, str(seed), "2000"], capture_output=True, text=True).stdout.split()
    assert text and text[0] == "ok", " ".join(text)
    assert min(map(int, text[1:])) > 100       # two products, units taken ahead, half units, split sums
