"""The example of the training operators together: its gradients against the binary64 oracle, and its
loss goes down."""

import os
import sys

import numpy as np
import pytest
import torch

import persistent_warp_specialized_gb300 as tg
from gpu_helpers import ensure_library
from oracle import train

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.fixture(scope="module", autouse=True)
def library():
    ensure_library()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_gradients_of_the_layer(dtype):
    import norm_linear_step as ex

    rows, cols, outs = 300, 264, 136
    gen = torch.Generator().manual_seed(3)
    x = (torch.randn((rows, cols), generator=gen) + 0.5).to(dtype)
    dz = (0.1 * torch.randn((rows, outs), generator=gen)).to(dtype)
    layer = ex.NormLinear(cols, outs, dtype)
    z, saved = layer.forward(x.cuda())
    dx, dgamma, dbeta, dw = layer.backward(dz.cuda(), saved)
    assert tg.tg_device_status() == 0

    x64, dz64 = x.double().numpy(), dz.double().numpy()
    w = layer.w.to(dtype).double().cpu().numpy()
    y, mean, rstd = train.norm(x64, np.ones(cols), np.zeros(cols), 1e-5)
    kept_x, kept_y = saved[0], saved[1]
    y8 = train.unpack(kept_y.q.cpu().numpy(), kept_y.s.cpu().numpy(), cols)
    x8 = train.unpack(kept_x.q.cpu().numpy(), kept_x.s.cpu().numpy(), cols)
    # 8 bits: half a step of E4M3's 3 fraction bits (1/16), saturation at most 1/8 of a block's top
    assert np.linalg.norm(y8 - y) < 0.05 * np.linalg.norm(y)
    half_ulp = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    near = lambda a, b: np.linalg.norm(a.double().cpu().numpy() - b) / np.linalg.norm(b)  # noqa: E731
    # each result: its inputs' and its own rounding, a few half ulps in the 2-norm
    assert near(z, y @ w) < 4 * half_ulp
    assert near(dw, y8.T @ dz64) < 4 * half_ulp
    rx, rg, rb = train.norm_backward(dz64 @ w.T, x8, mean, rstd, np.ones(cols))
    assert near(dx, rx) < 4 * half_ulp
    assert near(dgamma, rg) < 4 * half_ulp and near(dbeta, rb) < 4 * half_ulp


def test_the_loss_goes_down():
    import norm_linear_step as ex

    losses = ex.main(["--rows", "512", "--cols", "256", "--outs", "256", "--steps", "8"])
    assert losses[-1] < 0.5 * losses[0] and all(b < a for a, b in zip(losses, losses[1:]))
