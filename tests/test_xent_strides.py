"""Rows' values of any stride pass the checks of the Python layer (no GPU: the device is missed after them)."""

import pytest
import torch

import persistent_warp_specialized_gb300 as tg
from persistent_warp_specialized_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def library():
    _build.build()


def test_strides_are_not_refused():
    x, w = torch.zeros((4, 32), dtype=torch.bfloat16), torch.zeros((7, 32), dtype=torch.bfloat16)
    targets, lse = torch.zeros((4, 3), dtype=torch.int64)[:, 1], torch.zeros((4, 2))[:, 0]
    with pytest.raises(tg.TgError):
        tg.linear_cross_entropy(x, w, targets)
    for dloss in (torch.ones(()).expand(4), torch.ones((4, 2))[:, 1], torch.ones(4)):
        with pytest.raises(tg.TgError):
            tg.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    with pytest.raises(ValueError, match="4 values"):
        tg.linear_cross_entropy_backward(torch.ones(()).expand(5), x, w, targets, lse)
