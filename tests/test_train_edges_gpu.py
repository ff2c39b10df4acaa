"""Edges of the training operators: rows without columns, lanes without values, constant rows whose
value takes all of a float's bits, and matrices that lie in each other's gaps.  Tolerances:
test_norm_gpu.py."""

import numpy as np
import pytest
import torch

import persistent_warp_specialized_gb300 as tg
from gpu_helpers import ensure_library
from oracle import train
from test_norm_gpu import DT, check_backward, check_forward, f64, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    ensure_library()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_rows_without_columns(dtype):
    # the mean of no values is 0 / 0
    x = torch.empty((300, 0), dtype=DT[dtype], device="cuda")
    mean, rstd = (torch.full((300,), 7.0, device="cuda") for _ in range(2))
    tg.tg_layernorm_fwd(None, None, None, None, mean, rstd, None, None, 300, 0, 0, 0, dtype)
    assert torch.isnan(mean).all() and torch.isnan(rstd).all()
    mean.fill_(7.0)
    tg.tg_layernorm_fwd(None, None, None, None, mean, None, None, None, 300, 0, 0, 0, dtype)
    assert torch.isnan(mean).all()
    del mean, rstd                               # what torch.empty is likely to hand out next
    y, mean, rstd, kept = tg.layer_norm(x, checkpoint=True)
    assert y.shape == (300, 0) and (kept.rows, kept.cols) == (300, 0)
    assert torch.isnan(mean).all() and torch.isnan(rstd).all()
    dx, dgamma, dbeta = tg.layer_norm_backward(x, kept, mean, rstd)
    assert dx.shape == (300, 0) and dgamma.shape == dbeta.shape == (0,)


# A group's last lanes have no values at these widths.  The rows are constant and so large that
# mean * rstd is infinite, while every value's (x - mean) rstd is zero.
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("cols", [40, 136, 264, 520, 1000, 4104, 8200, 12296, 16392])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lanes_without_values_count_for_nothing(dtype, cols, kept):
    _, gamma, _, dy = make(5, cols, dtype, seed=cols)
    x = torch.full((5, cols), 2.0 ** 120, dtype=DT[dtype])
    mean, rstd = torch.full((5,), 2.0 ** 120), torch.full((5,), 2.0 ** 10)
    xd = tg.ckpt8_pack(x.cuda()) if kept else x.cuda()
    got = tg.layer_norm_backward(dy.cuda(), xd, mean.cuda(), rstd.cuda(), gamma.cuda())
    assert torch.isfinite(got[0]).all()
    check_backward(dy, f64(x), mean, rstd, gamma, got, dtype)
    assert (got[1] == 0).all()
