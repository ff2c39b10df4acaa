"""Layer norm where a group of threads takes several rows in turn, and where that is easiest to get
wrong: the sums over rows are exact integers here, so that a lost or repeated row shows whatever the
number of rows.  And the calls a training program makes around it: graphs, streams, threads.

Tolerances of what is not exact: test_norm_gpu.py.  Its comparisons pass over NaN, so every result is
asserted to be finite as well."""

import threading

import numpy as np
import pytest
import torch

import persistent_warp_specialized_gb300 as tg
from gpu_helpers import ensure_library
from oracle import train
from test_norm_gpu import DT, SHAPES, check_backward, check_forward, f64, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    ensure_library()


def offset_by(t, n, pad=0):
    """t in a larger buffer of NaN, its rows ``pad`` values apart, n values after a 16-byte boundary."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + 64,), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[16 + n:16 + n + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    return view.copy_(t)


# (rows, cols): at least three rows to each group of threads, and no whole number of turns
SHORT = [(9001, 64), (5003, 33), (12001, 100)]                    # rows of at most 512 bytes
LEAD = [(4001, 517), (700, 4099), (500, 8185)]                    # rows that start alike off the grid
GROUPED = [(8001, 264), (4001, 520), (1001, 4096), (500, 8192)]
WIDE = [(500, 8200), (500, 16384)]                                # 16 bits: 1024 threads; fp32: any width
LONG = [(300, 16392), (200, 20008)]
CASES = ([(r, c, "whole") for r, c in SHORT + LEAD + GROUPED + WIDE + LONG]
         + [(r, c, "any") for r, c in [(5003, 99), (4001, 520), (700, 4099), (500, 9001), (300, 16411)]]
         + [(r, c, "kept") for r, c in [(9001, 64), (5003, 99)] + GROUPED + WIDE + [(300, 16392)]]
         + [(r, c, "kept_any") for r, c in [(4001, 517), (700, 4099), (500, 9001), (300, 16411)]])


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols,form", CASES)
def test_sums_over_rows_are_exact(rows, cols, form, dtype):
    gen = torch.Generator().manual_seed(rows + cols)
    x = torch.randint(-4, 5, (rows, cols), generator=gen).to(DT[dtype])
    dy = torch.randint(-2, 3, (rows, cols), generator=gen).to(DT[dtype])
    gamma = 1 + 0.3 * torch.randn(cols, generator=gen)
    mean, rstd = torch.zeros(rows), torch.ones(rows)
    xd, dyd = x.cuda(), dy.cuda()
    if form == "any":                            # not alike in all tensors
        xd, dyd = offset_by(x, 1, pad=2), offset_by(dy, 3, pad=1)
    if form == "kept_any":
        dyd = offset_by(dy, 1, pad=3)
    if form.startswith("kept"):
        xd = tg.ckpt8_pack(x.cuda())
        assert torch.equal(tg.ckpt8_unpack(xd, DT[dtype]).cpu(), x)
    want = (dy.double() * x.double()).sum(dim=0), dy.double().sum(dim=0)
    first = None
    for _ in range(2):
        dx, dgamma, dbeta = tg.layer_norm_backward(dyd, xd, mean.cuda(), rstd.cuda(), gamma.cuda())
        assert torch.equal(dgamma.double().cpu(), want[0])
        assert torch.equal(dbeta.double().cpu(), want[1])
        assert first is None or torch.equal(dx, first)
        first = dx
    assert torch.isfinite(dx).all()
    check_backward(dy, f64(x), mean, rstd, gamma, (dx, dgamma, dbeta), dtype)


# Forward kernels by (rows, cols): 16 values a thread, whole rows and others; 1024 threads; fp32.
@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("rows,cols,dtype,form", [
    (7501, 1000, "bf16", "whole"), (2003, 4096, "f16", "whole"), (1703, 8192, "bf16", "whole"),
    (7501, 520, "f32", "whole"), (2003, 4096, "f32", "whole"), (1003, 8192, "f32", "whole"),
    (7001, 1001, "f16", "whole"), (2003, 4099, "f32", "whole"), (1501, 3001, "bf16", "any"),
    (1003, 4099, "f32", "any"), (607, 16384, "bf16", "whole"), (607, 9001, "f16", "any"),
    (501, 9000, "f32", "whole"), (501, 16383, "f32", "any"), (12001, 100, "f32", "any"),
    (12001, 200, "bf16", "whole"), (403, 16400, "f16", "whole")])
def test_forward_of_many_rows(rows, cols, dtype, form, checkpoint):
    x, gamma, beta, _ = make(rows, cols, dtype, seed=rows + cols)
    xd = offset_by(x, 3, pad=1) if form == "any" else x.cuda()
    got = tg.layer_norm(xd, gamma.cuda(), beta.cuda(), checkpoint=checkpoint)
    assert all(torch.isfinite(t).all() for t in got[:3])
    check_forward(x, gamma, beta, got[:3], dtype)
    again = tg.layer_norm(xd, gamma.cuda(), beta.cuda())
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    if checkpoint:
        q, s = train.pack(f64(got[0]))
        np.testing.assert_array_equal(got[3].s.cpu().numpy(), s)
        np.testing.assert_array_equal(got[3].q.cpu().numpy(), q)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_every_result_is_a_number(rows, cols, dtype):
    x, gamma, beta, dy = make(rows, cols, dtype, seed=rows + cols)
    y, mean, rstd, kept = tg.layer_norm(x.cuda(), gamma.cuda(), beta.cuda(), checkpoint=True)
    for t in (y, mean, rstd, tg.ckpt8_unpack(kept, DT[dtype])):
        assert torch.isfinite(t).all()
    kept = tg.ckpt8_pack(x.cuda())
    x8 = train.unpack(kept.q.cpu().numpy(), kept.s.cpu().numpy(), cols)
    for xd, x64 in ((x.cuda(), f64(x)), (kept, x8)):
        got = tg.layer_norm_backward(dy.cuda(), xd, mean, rstd, gamma.cuda())
        ref = train.norm_backward(f64(dy), x64, f64(mean), f64(rstd), f64(gamma))
        for t, r in zip(got, ref):   # an 8-bit value's distance from the mean times rstd^3 may leave fp16
            assert torch.equal(torch.isfinite(t).cpu(), torch.isfinite(torch.from_numpy(r).to(t.dtype)))


def step(x, gamma, beta, dy, stream=None):
    y, mean, rstd, kept = tg.layer_norm(x, gamma, beta, checkpoint=True, stream=stream)
    kept_x = tg.ckpt8_pack(x, stream=stream)
    dw = tg.ckpt8_wgrad(kept, dy, stream=stream)
    grads = tg.layer_norm_backward(dy, kept_x, mean, rstd, gamma, stream=stream)
    return (y, mean, rstd, kept.q, kept.s, dw, *grads)


def inputs(seed, rows=700, cols=1000, dtype="bf16"):
    return [t.cuda() for t in make(rows, cols, dtype, seed=seed)]


def test_a_step_in_a_graph_follows_its_inputs():
    x, gamma, beta, dy = inputs(0)
    step(x, gamma, beta, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, gamma, beta, dy)
    for seed in (1, 2, 3):
        others = inputs(seed)
        for t, other in zip((x, gamma, beta, dy), others):
            t.copy_(other)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, step(*others)))


def test_a_step_on_another_stream():
    args = inputs(4)
    want = step(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = step(*args, stream=stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_steps_from_several_threads():
    jobs = [inputs(10 + i, rows=300 + 70 * i, cols=264 * (i + 1)) for i in range(4)]
    want = [step(*job) for job in jobs]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(10):
                got = step(*jobs[i], stream=stream)
                stream.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        except BaseException as e:   # noqa: BLE001  (reported below)
            failed.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and tg.tg_device_status() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(700, 24), (700, 99), (900, 520), (900, 1001), (400, 4096),
                                       (400, 4099), (300, 8192), (200, 9001), (60, 16400),
                                       (3700, 4096)])
def test_a_row_gives_the_same_bits_wherever_it_lies(rows, cols, dtype):
    x, gamma, beta, _ = make(rows, cols, dtype, seed=cols)
    gd, bd = gamma.cuda(), beta.cuda()
    want = tg.layer_norm(x.cuda(), gd, bd, checkpoint=True)
    for n, pad in ((0, 8), (0, 3), (1, 0), (5, 2)):
        got = tg.layer_norm(offset_by(x, n, pad), gd, bd, checkpoint=n != 1)
        assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3])), (n, pad)
        if n != 1:
            assert torch.equal(got[3].q, want[3].q) and torch.equal(got[3].s, want[3].s)
