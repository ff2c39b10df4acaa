"""The fused products' host code built with g++ against stand-ins for the CUDA runtime and the kernels (no GPU):
random calls, with every tensor map and pointer that reaches a launch inside the buffers of the call, as
large as the workspace queries said, and every unit of work walked once."""

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
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(_build.nvcc())))),
                        "include")
    out = str(tmp_path_factory.mktemp("host") / "linear_host_driver")
    # kernels that no test reaches are left undefined
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", cuda, "-I", _build.CSRC, "-x", "c++",
                    os.path.join(ROOT, "tests", "linear_host_driver.cpp"),
                    os.path.join(_build.CSRC, "tg_api.cu"),
                    os.path.join(_build.CSRC, "tg_linear_api.cu"),
                    "-Wl,--unresolved-symbols=ignore-all", "-o", out], check=True)
    return out


@pytest.mark.parametrize("seed", range(4))
def test_every_launch_stays_in_its_buffers(driver, seed):
    text = subprocess.run([driver, str(seed), "1500"], capture_output=True, text=True).stdout.split()
    assert text and text[0] == "ok", " ".join(text)
    calls, launches, few, two, splits, groups, parts, pieces = map(int, text[1:])
    # every way is among them
    assert min(launches, few) > 200 and min(two, splits, parts) > 20 and min(groups, pieces) >= 3
