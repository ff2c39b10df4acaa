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


# The sum of equal values is rounded where they take all of a float's bits; their mean is the value.
@pytest.mark.parametrize("cols", [1, 3, 31, 100, 128, 129, 700, 1001, 4099, 5000, 8192, 9000, 16384,
                                  20000, 40001])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_constant_rows_of_any_value(cols, dtype):
    values = torch.tensor([0.1, 1.1, 1000.3, 1 / 3, -7.7, 1.0009765625]).to(DT[dtype])
    x = values[:, None].repeat(1, cols).cuda()
    y, mean, rstd = tg.layer_norm(x, eps=1e-5)
    assert torch.equal(mean.cpu(), values.float()) and (y == 0).all()
    torch.testing.assert_close(rstd.cpu(), torch.full((6,), 1e-5 ** -0.5), rtol=1e-6, atol=0)
    y, mean, _ = tg.layer_norm(x, eps=0.0)       # 0 times whatever the root's inverse is
    assert torch.equal(mean.cpu(), values.float()) and ((y == 0) | torch.isnan(y)).all()
    beta = torch.linspace(-2, 2, cols, device="cuda")
    y = tg.layer_norm(x, beta=beta, eps=1e-5)[0]
    assert torch.equal(y, beta.to(DT[dtype])[None].expand(6, cols))


# Deviations far below the mean: what is left of them is what the mean's own rounding leaves.
@pytest.mark.parametrize("cols", [100, 1000, 4099, 8192, 20000])
def test_small_deviations_about_a_large_mean(cols):
    gen = torch.Generator().manual_seed(cols)
    steps = torch.randint(-8, 9, (7, cols), generator=gen)
    x = 1000.3 + steps * 2.0 ** -14              # one to eight units in the last place
    _, mean, rstd = tg.layer_norm(x.float().cuda(), eps=1e-12)
    _, rm, rr = train.norm(f64(x.float()), None, None, 1e-12)
    # the mean to a unit in the last place, and the variance about it to one part in 100
    assert (np.abs(f64(mean) - rm) <= 2.0 ** -14).all()
    assert (np.abs(f64(rstd) / rr - 1) < 0.005).all()


# Column slices of one buffer: they share no element, whichever comes first.
@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("cols,gap,lead", [(48, 0, 0), (264, 3, 5), (700, 0, 8), (4096, 8, 0)])
def test_outputs_between_the_inputs_rows(cols, gap, lead, dtype):
    rows, ld = 37, lead + 2 * cols + gap
    x, gamma, beta, dy = make(rows, cols, dtype, seed=cols)
    gd, bd = gamma.cuda(), beta.cuda()
    for first in (0, 1):
        def slices():
            buf = torch.full((rows, ld), 7.0, dtype=DT[dtype], device="cuda")
            halves = buf[:, lead:lead + cols], buf[:, lead + cols:lead + 2 * cols]
            return buf, halves[first], halves[1 - first]

        def intact(buf):
            return (buf[:, :lead] == 7).all() and (buf[:, lead + 2 * cols:] == 7).all()

        buf, xs, y = slices()
        xs.copy_(x)
        got = tg.layer_norm(xs, gd, bd, out=y)
        check_forward(x, gamma, beta, got, dtype)
        assert torch.equal(xs.cpu(), x) and intact(buf)
        buf, dys, dx = slices()
        dys.copy_(dy)
        dgamma, dbeta = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        nbytes = tg.tg_layernorm_bwd_workspace_bytes(rows, cols)
        ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        tg.tg_layernorm_bwd(dys, x.cuda(), None, None, gd, got[1], got[2], dx, dgamma, dbeta, rows,
                            cols, ld, cols, ld, dtype, "f32", ws)
        check_backward(dy, f64(x), got[1], got[2], gamma, (dx, dgamma, dbeta), dtype)
        assert torch.equal(dys.cpu(), dy) and intact(buf)


def test_a_weight_gradient_between_its_inputs_rows():
    buf = torch.zeros((200, 256), dtype=torch.bfloat16, device="cuda")
    dy, dw = buf[:, :120], buf[:96, 136:]
    gen = torch.Generator().manual_seed(1)
    dy.copy_(torch.randint(-2, 3, (200, 120), generator=gen))
    x = torch.randint(-4, 5, (200, 96), generator=gen).float()
    tg.ckpt8_wgrad(tg.ckpt8_pack(x.cuda()), dy, out=dw)
    assert torch.equal(dw.cpu().double(), (x.double().T @ dy.cpu().double()).bfloat16().double())
    assert (buf[96:, 136:] == 0).all() and (buf[:, 120:136] == 0).all()


def test_outputs_that_do_overlap_are_refused():
    buf = torch.zeros((40, 256), dtype=torch.float16, device="cuda")
    flat = buf.view(-1)

    def refused(x, out):
        with pytest.raises(tg.TgError) as e:
            tg.layer_norm(x, out=out)
        assert e.value.code == tg.TG_ERR_ARG and "overlaps" in str(e.value)

    refused(buf[:, :128], buf[:, :128])
    refused(buf[:, :128], buf[:, 127:255])                     # one column
    refused(buf[:, 127:255], buf[:, :128])
    wrapped = flat[200:].as_strided((39, 100), (256, 1))       # columns 200 .. 255 and 0 .. 43
    refused(buf[:39, :100], wrapped)
    refused(wrapped, buf[:39, :100])
    refused(wrapped, buf[:39, 101:201])
    tg.layer_norm(buf[:39, 60:160], out=wrapped)               # between 44 and 199
    tg.layer_norm(wrapped, out=buf[:39, 60:160])
    refused(buf[:20, :64], flat[64:].as_strided((20, 64), (512, 1)))      # rows of another pitch
    refused(buf[:, :64], flat[64:64 + 40 * 64].view(40, 64))
    tg.layer_norm(buf[:20, :128], out=buf[20:, :128])          # one after the other
    tg.layer_norm(flat[:256].view(1, 256), out=flat[256:512].view(1, 256))
    mean = torch.zeros(40, device="cuda")
    y = torch.empty((40, 128), dtype=torch.float16, device="cuda")
    with pytest.raises(tg.TgError):
        tg.tg_layernorm_fwd(buf[:, :128], None, None, y, y.view(torch.float32)[0], mean, None, None,
                            40, 128, 256, 128, "f16")
