"""Layer norm forward and backward against the binary64 oracle.

Tolerances, fixed before the first run, with u = 2^-24:
  * a sum of n fp32 terms taken in any tree of depth d is off by at most d u times the sum of
    magnitudes; the kernels' trees over a row are at most 64 deep (values in a thread, lanes, warps)
    below 16384 columns, and cols / 1024 + 64 deep above;
  * what follows a sum adds a few roundings; 16 are allowed;
  * the result is rounded once to its type: half an ulp.
"""

import numpy as np
import pytest
import torch

import persistent_warp_specialized_gb300 as tg
from gpu_helpers import ensure_library
from oracle import train

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF_ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # relative, normal numbers
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}    # half the subnormal step


@pytest.fixture(scope="module", autouse=True)
def library():
    ensure_library()


def rounding(v, dtype):
    return np.abs(v) * HALF_ULP[dtype] + TINY[dtype]


def depth(cols):
    return 64 + (cols // 1024 if cols > 16384 else 0) + 16


def make(rows, cols, dtype, seed=0, mean=0.3, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=gen) * scale * torch.exp(
        0.5 * torch.randn(cols, generator=gen)) + mean
    gamma = 1 + 0.3 * torch.randn(cols, generator=gen)
    beta = 0.3 * torch.randn(cols, generator=gen)
    dy = torch.randn((rows, cols), generator=gen)
    return x.to(DT[dtype]), gamma, beta, dy.to(DT[dtype])


def f64(t):
    return t.detach().cpu().double().numpy()


def check_forward(x, gamma, beta, got, dtype, eps=1e-5):
    y, mean, rstd = got
    xx = f64(x)
    g = None if gamma is None else f64(gamma)
    b = None if beta is None else f64(beta)
    ry, rm, rr = train.norm(xx, g, b, eps)
    d = depth(x.shape[1])
    size = np.abs(xx).mean(axis=1)                     # of the terms of the mean's sum
    assert (np.abs(f64(mean) - rm) <= d * U * size + U * np.abs(rm)).all()
    # the mean's error shifts every deviation; squares double relative errors, the root halves them
    shift = d * U * size * rr
    assert (np.abs(f64(rstd) - rr) <= rr * (d * U + 2 * shift)).all()
    xh = (xx - rm[:, None]) * rr[:, None]
    gg = np.ones(x.shape[1]) if g is None else np.abs(g)
    bb = np.zeros(x.shape[1]) if b is None else np.abs(b)
    tol = gg * (np.abs(xh) * (d * U + 2 * shift[:, None]) + shift[:, None] + 4 * U * np.abs(xh))
    tol = tol + 4 * U * bb
    err = np.abs(f64(y) - ry)
    bad = err > tol + rounding(np.abs(ry) + tol, dtype)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), err.max())


def check_backward(dy, x64, mean, rstd, gamma, got, dtype, param="f32"):
    dx, dgamma, dbeta = got
    rows, cols = dy.shape
    d64, m, r = f64(dy), f64(mean), f64(rstd)
    g64 = None if gamma is None else f64(gamma)
    rx, rg, rb = train.norm_backward(d64, x64, m, r, g64)
    xh = (x64 - m[:, None]) * r[:, None]
    g = np.abs(d64 * (1 if g64 is None else g64))
    d = depth(cols)
    parts = g.mean(axis=1, keepdims=True), (g * np.abs(xh)).mean(axis=1, keepdims=True)
    tol = r[:, None] * (d * U * (parts[0] + np.abs(xh) * parts[1]) +
                        8 * U * (g + parts[0] + np.abs(xh) * parts[1]))
    err = np.abs(f64(dx) - rx)
    bad = err > tol + rounding(np.abs(rx) + tol, dtype)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), err.max())
    for name, v, ref, mag in (("dgamma", dgamma, rg, np.abs(d64 * xh).sum(axis=0)),
                              ("dbeta", dbeta, rb, np.abs(d64).sum(axis=0))):
        tol = (rows + 16) * U * mag                    # any order of the rows
        err = np.abs(f64(v) - ref)
        assert (err <= tol + rounding(np.abs(ref) + tol, param)).all(), (name, err.max())


SHAPES = [(1, 1), (3, 1), (1, 7), (5, 8), (2, 31), (7, 33), (4, 64), (9, 255), (33, 256), (6, 257),
          (300, 512), (5, 1000), (17, 1024), (4, 1025), (3, 2047), (160, 4096), (2, 8191), (3, 8192),
          (2, 8200), (2, 16384), (1, 16392), (1, 40001)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, dtype):
    x, gamma, beta, _ = make(rows, cols, dtype, seed=rows * 7 + cols)
    got = tg.layer_norm(x.cuda(), gamma.cuda(), beta.cuda())
    check_forward(x, gamma, beta, got, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(rows, cols, dtype):
    x, gamma, beta, dy = make(rows, cols, dtype, seed=rows * 5 + cols)
    _, mean, rstd = tg.layer_norm(x.cuda(), gamma.cuda(), beta.cuda())
    got = tg.layer_norm_backward(dy.cuda(), x.cuda(), mean, rstd, gamma.cuda())
    check_backward(dy, f64(x), mean, rstd, gamma, got, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 33), (200, 512), (3, 2047), (40, 4096), (2, 8200)])
def test_backward_from_a_checkpoint(rows, cols, dtype):
    x, gamma, beta, dy = make(rows, cols, dtype, seed=rows * 3 + cols)
    _, mean, rstd = tg.layer_norm(x.cuda(), gamma.cuda(), beta.cuda())
    kept = tg.ckpt8_pack(x.cuda())
    got = tg.layer_norm_backward(dy.cuda(), kept, mean, rstd, gamma.cuda())
    x64 = train.unpack(kept.q.cpu().numpy(), kept.s.cpu().numpy(), cols)
    check_backward(dy, x64, mean, rstd, gamma, got, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 31), (9, 200), (7, 1000), (3, 2047), (4, 4096),
                                       (1, 16392)])
def test_forward_keeps_a_checkpoint_of_what_it_wrote(rows, cols, dtype):
    x, gamma, beta, _ = make(rows, cols, dtype, seed=cols)
    y, mean, rstd, kept = tg.layer_norm(x.cuda(), gamma.cuda(), beta.cuda(), checkpoint=True)
    check_forward(x, gamma, beta, (y, mean, rstd), dtype)
    q, s = train.pack(f64(y))
    np.testing.assert_array_equal(kept.s.cpu().numpy(), s)
    np.testing.assert_array_equal(kept.q.cpu().numpy(), q)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("with_gamma,with_beta", [(False, False), (True, False), (False, True)])
def test_parameters_may_be_absent_or_of_the_values_type(dtype, with_gamma, with_beta):
    x, gamma, beta, dy = make(37, 520, dtype, seed=5)
    gamma = gamma.to(DT[dtype]) if with_gamma else None
    beta = beta.to(DT[dtype]) if with_beta else None
    dev = [None if t is None else t.cuda() for t in (gamma, beta)]
    got = tg.layer_norm(x.cuda(), *dev)
    check_forward(x, gamma, beta, got, dtype)
    grads = tg.layer_norm_backward(dy.cuda(), x.cuda(), got[1], got[2], dev[0])
    check_backward(dy, f64(x), got[1], got[2], gamma, grads, dtype, dtype if with_gamma else "f32")


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("offset,pad", [(0, 8), (0, 3), (1, 0), (3, 5), (8, 16)])
def test_row_strides_and_unaligned_bases(dtype, offset, pad):
    rows, cols = 19, 712
    x, gamma, beta, dy = make(rows, cols, dtype, seed=offset + pad)

    def strided(t):
        flat = torch.full((offset + rows * (cols + pad),), float("nan"), dtype=t.dtype, device="cuda")
        v = flat[offset:].view(rows, cols + pad)[:, :cols]
        v.copy_(t)
        return v

    xs, dys, out = strided(x), strided(dy), strided(torch.zeros_like(x))
    gs, bs = gamma.cuda(), beta.cuda()
    got = tg.layer_norm(xs, gs, bs, out=out)
    check_forward(x, gamma, beta, got, dtype)
    whole = out.as_strided((rows, cols + pad), (cols + pad, 1))
    assert torch.isnan(whole[:rows - 1, cols:]).all()      # nothing is written between the rows
    grads = tg.layer_norm_backward(dys, xs, got[1], got[2], gs)
    check_backward(dy, f64(x), got[1], got[2], gamma, grads, dtype)
    # parameters off the 16-byte grid
    g1 = torch.cat([torch.zeros(1), gamma]).cuda()[1:]
    b1 = torch.cat([torch.zeros(1), beta]).cuda()[1:]
    check_forward(x, gamma, beta, tg.layer_norm(xs, g1, b1), dtype)


@pytest.mark.parametrize("rows,cols", [(4, 300), (2, 4096), (1, 20000)])
def test_a_large_mean_costs_no_digits(rows, cols):
    # deviations of 1 about a mean of 1000: sum x^2 - (sum x)^2 would lose six digits
    x, gamma, beta, _ = make(rows, cols, "f32", seed=9, mean=1000.0)
    check_forward(x, gamma, beta, tg.layer_norm(x.cuda(), gamma.cuda(), beta.cuda()), "f32")


@pytest.mark.parametrize("cols", [5, 700, 5000, 20000])
def test_constant_rows(cols):
    x = torch.full((3, cols), 2.5)
    y, mean, rstd = tg.layer_norm(x.cuda(), eps=1e-5)
    assert (mean == 2.5).all() and (y == 0).all()
    torch.testing.assert_close(rstd.cpu(), torch.full((3,), 1e-5 ** -0.5), rtol=1e-6, atol=0)
    y0, _, rstd0 = tg.layer_norm(x.cuda(), eps=0.0)       # 0 * inf, as the formula says
    assert torch.isinf(rstd0).all() and torch.isnan(y0).all()


@pytest.mark.parametrize("cols", [40, 1000, 4096, 20000])
def test_what_is_not_finite_stays_in_its_row(cols):
    x, gamma, beta, dy = make(6, cols, "bf16", seed=3)
    x[1, cols // 2] = float("nan")
    x[3, 0] = float("inf")
    dy[4, cols - 1] = float("nan")
    y, mean, rstd = tg.layer_norm(x.cuda(), gamma.cuda(), beta.cuda())
    bad = [1, 3]
    fine = [0, 2, 4, 5]
    assert torch.isnan(y[bad]).all()
    check_forward(x[fine], gamma, beta, (y[fine], mean[fine], rstd[fine]), "bf16")
    dx, dgamma, dbeta = tg.layer_norm_backward(dy.cuda(), x.cuda(), mean, rstd, gamma.cuda())
    assert torch.isnan(dx[[1, 3, 4]]).all() and torch.isnan(dgamma).all()
    assert torch.isfinite(dx[[0, 2, 5]].float()).all()
    assert torch.isnan(dbeta).nonzero().flatten().tolist() == [cols - 1]


def test_no_rows():
    x = torch.empty((0, 48), device="cuda")
    y, mean, rstd = tg.layer_norm(x)
    assert y.shape == (0, 48) and mean.shape == (0,)
    dx, dgamma, dbeta = tg.layer_norm_backward(x, x, mean, rstd)
    assert dx.shape == (0, 48) and (dgamma == 0).all() and (dbeta == 0).all()


def test_more_rows_than_a_wave_and_repeatable_sums():
    x, gamma, beta, dy = make(5003, 264, "bf16", seed=11)
    _, mean, rstd = tg.layer_norm(x.cuda(), gamma.cuda(), beta.cuda())
    first = tg.layer_norm_backward(dy.cuda(), x.cuda(), mean, rstd, gamma.cuda())
    check_backward(dy, f64(x), mean, rstd, gamma, first, "bf16")
    for _ in range(3):
        again = tg.layer_norm_backward(dy.cuda(), x.cuda(), mean, rstd, gamma.cuda())
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_offsets_past_32_bits():
    # 70000 rows of 65536 values: 4.6e9 elements, 18 GB
    rows, cols = 70000, 65536
    x = torch.zeros((rows, cols), dtype=torch.float16, device="cuda")
    part, gamma, beta, dyp = make(3, cols, "f16", seed=4)
    at = [0, 32768, rows - 1]                              # 32768 * 65536 = 2^31
    x[at] = part.cuda()
    y, mean, rstd, kept = tg.layer_norm(x, gamma.cuda(), beta.cuda(), checkpoint=True)
    check_forward(part, gamma, beta, (y[at], mean[at], rstd[at]), "f16")
    q, s = train.pack(f64(y[at]))
    np.testing.assert_array_equal(kept.q[at].cpu().numpy(), q)
    np.testing.assert_array_equal(kept.s[at].cpu().numpy(), s)
    assert (y[5] == beta.half().cuda()).all()
    dy = torch.zeros_like(x)
    dy[at] = dyp.cuda()
    dx, dgamma, dbeta = tg.layer_norm_backward(dy, x, mean, rstd, gamma.cuda())
    check_backward(dyp, f64(part), mean[at], rstd[at], gamma, (dx[at], dgamma, dbeta), "f16")


def test_another_stream():
    x, gamma, beta, dy = make(700, 2048, "bf16", seed=8)
    xd, gd, bd, dyd = (t.cuda() for t in (x, gamma, beta, dy))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = tg.layer_norm(xd, gd, bd, stream=stream)
        grads = tg.layer_norm_backward(dyd, xd, got[1], got[2], gd, stream=stream)
        side.synchronize()
        check_forward(x, gamma, beta, got, "bf16")
        check_backward(dy, f64(x), got[1], got[2], gamma, grads, "bf16")


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(2, 31), (3, 7), (5, 255), (4, 257), (7, 1001), (3, 4099),
                                       (2, 9001), (2, 16387)])
@pytest.mark.parametrize("offset", [0, 1, 5])
def test_nothing_is_written_outside(rows, cols, dtype, offset):
    # y, dx and unpacked values inside larger buffers: the 300 values before and after stay
    x, gamma, beta, dy = make(rows, cols, dtype, seed=cols)
    dev = [t.cuda() for t in (x, gamma, beta, dy)]
    n = rows * cols

    def guarded():
        buf = torch.full((n + 600 + offset,), 7.0, dtype=DT[dtype], device="cuda")
        return buf, buf[300 + offset:300 + offset + n].view(rows, cols)

    def intact(buf):
        return (buf[:300 + offset] == 7).all() and (buf[300 + offset + n:] == 7).all()

    buf, y = guarded()
    got = tg.layer_norm(*dev[:3], out=y)
    check_forward(x, gamma, beta, got, dtype)
    assert intact(buf)
    buf, dx = guarded()
    dgamma, dbeta = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(tg.tg_layernorm_bwd_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    tg.tg_layernorm_bwd(dev[3], dev[0], None, None, dev[1], got[1], got[2], dx, dgamma, dbeta, rows,
                        cols, cols, cols, cols, dtype, "f32", ws)
    check_backward(dy, f64(x), got[1], got[2], gamma, (dx, dgamma, dbeta), dtype)
    assert intact(buf)
    buf, out = guarded()
    kept = tg.ckpt8_pack(dev[0])
    tg.ckpt8_unpack(kept, DT[dtype], out=out)
    v = train.unpack(kept.q.cpu().numpy(), kept.s.cpu().numpy(), cols)
    assert torch.equal(out.cpu(), torch.from_numpy(v).to(DT[dtype])) and intact(buf)


# From 96 Ki values an SM on, 16-bit rows of 2049 to 16384 values go 32 to a thread.
@pytest.mark.parametrize("dtype,param", [("f16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,cols,pad", [(7400, 2049, 0), (5001, 3001, 3), (3700, 4096, 0),
                                           (2200, 7000, 8), (1900, 8192, 0), (1830, 8199, 0),
                                           (950, 16383, 1), (950, 16384, 0)])
def test_many_long_rows(rows, cols, pad, dtype, param):
    part, gamma, beta, _ = make(61, cols, dtype, seed=cols)
    gamma, beta = gamma.to(DT[param]), beta.to(DT[param])
    at = torch.arange(rows) * 7 % 61                       # row r holds row at[r] of ``part``
    x = torch.zeros((rows, cols + pad), dtype=DT[dtype], device="cuda")[:, :cols]
    x.copy_(part[at].cuda())
    buf = torch.full((rows * cols + 602,), 7.0, dtype=DT[dtype], device="cuda")
    y = buf[301:-301].view(rows, cols)
    _, mean, rstd = tg.layer_norm(x, gamma.cuda(), beta.cuda(), out=y)
    assert (buf[:301] == 7).all() and (buf[-301:] == 7).all()
    again = tg.layer_norm(x, gamma.cuda(), beta.cuda(), checkpoint=True)
    first = torch.tensor([(at == r).nonzero()[0].item() for r in range(61)])
    check_forward(part, gamma, beta, (y[first], mean[first], rstd[first]), dtype)
    same = first[at].cuda()
    for got in (y, mean, rstd):
        assert torch.equal(got, got[same])
    assert all(torch.equal(a, b) for a, b in zip(again[:3], (y, mean, rstd)))
    kept = again[3]
    q, s = train.pack(f64(y[first]))
    np.testing.assert_array_equal(kept.q[first].cpu().numpy(), q)
    np.testing.assert_array_equal(kept.s[first].cpu().numpy(), s)
    assert torch.equal(kept.q, kept.q[same]) and torch.equal(kept.s, kept.s[same])


# Rows of at most 512 bytes, several to a warp: full and partial turns, each access width (16 bytes, 4,
# one value), x and dy with gaps between rows.
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 3, 0), (37, 17, 1), (5003, 20, 0), (4999, 24, 8),
                                           (5001, 33, 0), (9001, 64, 0), (3001, 90, 2),
                                           (4003, 128, 0), (2501, 129, 3), (5003, 200, 0),
                                           (3000, 254, 4), (5003, 256, 0)])
def test_short_rows(rows, cols, pad, dtype):
    x, gamma, beta, dy = make(rows, cols, dtype, seed=cols)
    xd, dyd = (torch.full((rows, cols + pad), 9.0, dtype=DT[dtype], device="cuda")[:, :cols]
               for _ in range(2))
    xd.copy_(x.cuda())
    dyd.copy_(dy.cuda())
    gd, bd = gamma.cuda(), beta.cuda()
    buf = torch.full((rows * cols + 600,), 7.0, dtype=DT[dtype], device="cuda")
    y = buf[300:-300].view(rows, cols)
    _, mean, rstd = tg.layer_norm(xd, gd, bd, out=y)
    assert (buf[:300] == 7).all() and (buf[-300:] == 7).all()
    check_forward(x, gamma, beta, (y, mean, rstd), dtype)
    y2, mean2, rstd2, kept = tg.layer_norm(xd, gd, bd, checkpoint=True)
    assert torch.equal(y2, y) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
    q, s = train.pack(f64(y))
    np.testing.assert_array_equal(kept.s.cpu().numpy(), s)
    np.testing.assert_array_equal(kept.q.cpu().numpy(), q)
    grads = tg.layer_norm_backward(dyd, xd, mean, rstd, gd)
    check_backward(dy, f64(x), mean, rstd, gamma, grads, dtype)
    again = tg.layer_norm_backward(dyd, xd, mean, rstd, gd)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    kept = tg.ckpt8_pack(xd)
    grads = tg.layer_norm_backward(dyd, kept, mean, rstd, gd)
    x64 = train.unpack(kept.q.cpu().numpy(), kept.s.cpu().numpy(), cols)
    check_backward(dy, x64, mean, rstd, gamma, grads, dtype)


def test_what_is_not_finite_stays_in_its_short_row():
    x, gamma, beta, _ = make(2000, 72, "bf16", seed=9)
    x[7, 3] = float("nan")
    x[40, 71] = float("-inf")
    xd = x.cuda()
    y, mean, rstd = tg.layer_norm(xd, gamma.cuda(), beta.cuda())
    fine = [r for r in range(2000) if r not in (7, 40)]
    assert torch.isnan(y[[7, 40]]).all()
    check_forward(x[fine], gamma, beta, (y[fine], mean[fine], rstd[fine]), "bf16")


# Rows that start inside a 16-byte granule, equally in all tensors; every tensor inside a larger
# buffer whose other values (NaN among the inputs, 7 among the outputs) must not matter and stay.
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,offset", [(1, 301, 0, 1), (3, 1023, 0, 0), (700, 517, 0, 3),
                                                  (1001, 2047, 0, 0), (2003, 1030, 3, 5),
                                                  (153, 4099, 0, 7), (500, 7001, 1, 2),
                                                  (305, 8185, 0, 1), (5003, 264, 1, 0)])
def test_rows_with_one_lead(rows, cols, pad, offset, dtype):
    x, gamma, beta, dy = make(rows, cols, dtype, seed=cols)
    ld, n = cols + pad, rows * (cols + pad)

    def inside(t, fill):
        buf = torch.full((n + 64 + offset,), fill, dtype=DT[dtype], device="cuda")
        m = buf[32 + offset:32 + offset + n].view(rows, ld)[:, :cols]
        if t is not None:
            m.copy_(t.cuda())
        return buf, m

    def intact(buf):
        gaps = buf[32 + offset:32 + offset + n].view(rows, ld)[:, cols:]
        return all((v == 7).all() for v in (buf[:32 + offset], buf[32 + offset + n:], gaps))

    gd, bd = gamma.cuda(), beta.cuda()
    xd, dyd = inside(x, float("nan"))[1], inside(dy, float("nan"))[1]
    buf, y = inside(None, 7.0)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    tg.tg_layernorm_fwd(xd, gd, bd, y, mean, rstd, None, None, rows, cols, ld, ld, dtype)
    check_forward(x, gamma, beta, (y, mean, rstd), dtype)
    assert intact(buf)
    ws = torch.empty(tg.tg_layernorm_bwd_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    grads = []
    for _ in range(2):
        buf, dx = inside(None, 7.0)
        dgamma, dbeta = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        tg.tg_layernorm_bwd(dyd, xd, None, None, gd, mean, rstd, dx, dgamma, dbeta, rows, cols, ld,
                            ld, ld, dtype, "f32", ws)
        check_backward(dy, f64(x), mean, rstd, gamma, (dx, dgamma, dbeta), dtype)
        assert intact(buf)
        grads.append((dx, dgamma, dbeta))
    assert all(torch.equal(a, b) for a, b in zip(*grads))
