"""The oracle of the training operators, pinned without the library: the formats' published values,
torch's float8 conversion, brute-force rounding, and gradients against differences."""

import numpy as np
import pytest
import torch

from oracle import train


def test_e4m3_values_are_the_formats():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(train.E4M3, v)
    assert train.E4M3[0x7E] == 448 and train.E4M3[0x01] == 2.0 ** -9 and np.isnan(train.E4M3[0x7F])


def test_to_e4m3_rounds_to_nearest_even():
    # every midpoint, and its float neighbours, against torch's conversion
    grid = train.E4M3[:127]
    mid = (grid[1:] + grid[:-1]) / 2
    v = np.concatenate([grid, mid, np.nextafter(mid.astype(np.float32), np.float32(0)),
                        np.nextafter(mid.astype(np.float32), np.float32(1e9))])
    v = np.concatenate([v, -v])
    want = torch.tensor(v, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(train.to_e4m3(v), want)
    np.testing.assert_array_equal(train.to_e4m3(np.array([449.0, 511.0, -1e30])), [0x7E, 0x7E, 0xFE])


@pytest.mark.parametrize("cols", [1, 31, 32, 33, 100])
def test_pack_scales_by_the_blocks_largest(cols):
    rng = np.random.default_rng(cols)
    x = rng.standard_normal((5, cols)) * np.exp2(rng.integers(-30, 30, size=(5, cols)))
    x[2] = 0.0
    q, s = train.pack(x)
    v = train.unpack(q, s, cols)
    assert (q[:, cols:] == 0).all() and (s[2] == 0).all() and (v[2] == 0).all()
    for r in range(5):
        for j in range(s.shape[1]):
            block = x[r, 32 * j:32 * j + 32]
            top = np.abs(block).max()
            if top == 0:
                continue
            unit = 2.0 ** (int(s[r, j]) - 127)
            assert 256 * unit <= top < 512 * unit
            # half a step of the E4M3 grid, or what saturation takes from values over 448
            err = np.abs(v[r, 32 * j:32 * j + 32] - block)
            assert (err <= np.maximum(np.abs(block) / 16, unit * 2.0 ** -10) + unit * 64 *
                    (np.abs(block) > 448 * unit)).all()


def test_pack_keeps_what_is_not_finite_as_nan():
    x = np.ones((1, 64))
    x[0, 3], x[0, 5], x[0, 40] = np.nan, np.inf, -np.inf
    q, s = train.pack(x)
    v = train.unpack(q, s, 64)
    assert np.isnan(v[0, [3, 5, 40]]).all() and np.nansum(v) == 61


def test_norm_gradients_against_differences():
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((4, 7)) + 0.5, rng.standard_normal((4, 7))
    gamma, beta = rng.standard_normal(7), rng.standard_normal(7)

    def loss(x, gamma, beta):
        return (train.norm(x, gamma, beta, 1e-5)[0] * dy).sum()

    _, mean, rstd = train.norm(x, gamma, beta, 1e-5)
    dx, dgamma, dbeta = train.norm_backward(dy, x, mean, rstd, gamma)
    h = 1e-6
    for grad, at in ((dx, 0), (dgamma, 1), (dbeta, 2)):
        args = [x, gamma, beta]
        for i in np.ndindex(grad.shape):
            step = np.zeros_like(args[at])
            step[i] = h
            up, down = list(args), list(args)
            up[at], down[at] = args[at] + step, args[at] - step
            # central differences: O(h^2) and the roundoff of a sum of about 30 terms over 2 h
            assert abs((loss(*up) - loss(*down)) / (2 * h) - grad[i]) < 1e-7


def test_weight_gradient_against_differences():
    rng = np.random.default_rng(2)
    q, s = train.pack(rng.standard_normal((6, 5)))
    dy, w = rng.standard_normal((6, 3)), rng.standard_normal((5, 3))
    x = train.unpack(q, s, 5)
    dw = train.weight_gradient(q, s, 5, dy)
    for i in np.ndindex(dw.shape):
        step = np.zeros_like(w)
        step[i] = 1.0
        assert abs((((x @ (w + step)) - (x @ w)) * dy).sum() - dw[i]) < 1e-12
