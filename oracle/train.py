"""Oracle of the training operators: layer norm and its gradients, 8-bit checkpoints, and the
weight gradient taken from a checkpoint, in binary64 numpy straight from their definitions.

A checkpoint of x [rows, cols] is (q, s): E4M3 bytes [rows, 32 ceil(cols / 32)], zero past ``cols``,
and E8M0 bytes [rows, ceil(cols / 32)]; it stands for q * 2^(s - 127).
"""

import numpy as np

BLOCK = 32


def e4m3_values():
    """The value of every E4M3 byte (1 sign, 4 exponent bits with bias 7, 3 fraction bits; exponent
    15 with fraction 7 is NaN, and there is no infinity)."""
    b = np.arange(256)
    e, f = (b >> 3) & 15, (b & 7).astype(np.float64)
    mag = np.where(e > 0, (1 + f / 8) * np.exp2(e - 7.0), f / 8 * 2.0 ** -6)
    mag[(e == 15) & (f == 7)] = np.nan
    return np.where(b >> 7, -mag, mag)


E4M3 = e4m3_values()


def to_e4m3(v):
    """Finite values -> E4M3 bytes: nearest, ties to the even byte, saturating at 448."""
    grid = E4M3[:127]                       # 0 .. 448, ascending
    a = np.minimum(np.abs(v), 448.0)
    hi = np.searchsorted(grid, a)           # grid[hi - 1] < a <= grid[hi]
    lo = np.maximum(hi - 1, 0)
    below, above = a - grid[lo], grid[hi] - a
    pick = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    return (pick | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def pack(x):
    """The checkpoint (q, s) of x (any float array [rows, cols]); NaN and infinities become NaN."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    b = np.zeros((rows, nb * BLOCK))
    b[:, :cols] = x
    b = b.reshape(rows, nb, BLOCK)
    fine = np.isfinite(b)
    amax = np.where(fine, np.abs(b), 0.0).max(axis=2, initial=0.0)
    e = np.where(amax > 0, np.frexp(amax)[1] - 1 - 8, -127).clip(-127, 127)
    q = to_e4m3(np.where(fine, b, 0.0) * np.exp2(-e.astype(np.float64))[:, :, None])
    q = np.where(fine, q, 0x7F).astype(np.uint8)
    return q.reshape(rows, nb * BLOCK), (e + 127).astype(np.uint8)


def unpack(q, s, cols):
    """The values (binary64, exact) that a checkpoint stands for; scale 255 is NaN."""
    scale = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
    return (E4M3[q] * np.repeat(scale, BLOCK, axis=1))[:, :cols]


def norm(x, gamma, beta, eps):
    """(y, mean, rstd) of layer norm over the rows of x; gamma and beta may be None."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * np.asarray(gamma, dtype=np.float64)
    if beta is not None:
        y = y + np.asarray(beta, dtype=np.float64)
    return y, mean, rstd


def norm_backward(dy, x, mean, rstd, gamma):
    """(dx, dgamma, dbeta) of ``norm`` at the statistics given."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    mean, rstd = np.asarray(mean, np.float64)[:, None], np.asarray(rstd, np.float64)[:, None]
    xh = (x - mean) * rstd
    g = dy if gamma is None else dy * np.asarray(gamma, dtype=np.float64)
    c1 = g.mean(axis=1, keepdims=True)
    c2 = (g * xh).mean(axis=1, keepdims=True)
    return rstd * (g - c1 - xh * c2), (dy * xh).sum(axis=0), dy.sum(axis=0)


def weight_gradient(q, s, cols, dy):
    """dW [cols, outs] = x^T dy for the x that the checkpoint stands for."""
    return unpack(q, s, cols).T @ np.asarray(dy, dtype=np.float64)
