"""The gated projections' gradients in fp16, whose products dh u act'(g) and dh act(g) leave its range at either
end while the gradients made of them do not."""

import pytest
import torch

import fused_ref as ref
import persistent_warp_specialized_gb300 as tg
from gpu_helpers import ensure_library

pytestmark = pytest.mark.gpu
F16 = torch.float16


@pytest.fixture(scope="module", autouse=True)
def library():
    ensure_library()


def exact(dh, g, u, x, wg, wu, act):
    dh, g, u, x, wg, wu = (t.double() for t in (dh, g, u, x, wg, wu))
    a, slope = ref.gate(g, act)
    dg, du = dh * u * slope, dh * a
    return {"dx": dg @ wg.t() + du @ wu.t(), "dwg": x.t() @ dg, "dwu": x.t() @ du}, max(dg.abs().max(), du.abs().max())


def problem(rows, cols, outs, dh, u, x, w, seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, scale):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(F16)

    return (normal((rows, outs), dh), normal((rows, outs), 1.5), normal((rows, outs), u), normal((rows, cols), x),
            normal((cols, outs), w), normal((cols, outs), w))


def far(got, want):
    """Distance in norm; a result below fp16's normal numbers may be off by half their step besides."""
    left = (got.double() - want).norm() - 2.0 ** -25 * want.numel() ** 0.5
    return float(left / want.norm())


# one row, two terms, few rows, the pair kernel, split sums; scales of dh, u, x and the weights that keep the
# gradients themselves in range
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,cols,outs", [(1, 136, 2056), (5, 264, 1000), (40, 264, 2056), (333, 1000, 2008),
                                            (2000, 264, 1288)])
@pytest.mark.parametrize("dh,u,x,w", [(1e-6, 0.1, 60.0, 60.0), (2e-5, 0.05, 30.0, 30.0), (1e-3, 1.0, 2.0, 2.0),
                                      (0.1, 1.0, 1.0, 0.02), (30.0, 30.0, 1e-2, 1e-3), (8e3, 20.0, 1e-3, 1e-4)])
def test_gradients_of_any_size(rows, cols, outs, dh, u, x, w, act):
    """dg and du are rounded once and the results once: a rounding is off by at most 2^-11 of its value, at random
    2^-11 / sqrt(3), so both together by 2^-11 sqrt(2 / 3) in norm."""
    args = problem(rows, cols, outs, dh, u, x, w)
    want, top = exact(*args, act)
    got = dict(zip(want, tg.gated_backward(*args, act=act)))
    torch.cuda.synchronize()
    assert tg.tg_device_status() == 0
    for name in want:
        assert want[name].abs().max() < 60000
        assert torch.isfinite(got[name]).all(), (name, float(top))
        assert far(got[name], want[name]) <= 2.0 ** -11, (name, far(got[name], want[name]), float(top))


@pytest.mark.parametrize("rows", [10, 60, 300])
def test_small_rows_beside_large_ones(rows):
    """Each row's dx keeps its bits beside rows 2^10 times as large.  What is added to the two roundings is the
    smallest step of dg and du: half of 2^-24, at a scale of 2^4 where the largest, scaled, is in [4, 65504],
    and else at one that takes it to 2^14 at least."""
    dh, g, u, x, wg, wu = problem(rows, 264, 1000, 1.0, 1.0, 1.0, 1.0, seed=2)
    scale = 2.0 ** -(torch.arange(rows, device="cuda") % 3 * 5).float()[:, None]
    for largest in (2.0 ** -6, 1.0, 2.0 ** 8):
        args = (dh.float() * scale * largest).half(), g, u, x, (wg / largest ** 0.5).half(), (wu / largest ** 0.5).half()
        want, top = exact(*args, "silu")
        half_step = 2.0 ** -29 if 4 <= 16 * top <= 65504 else float(top) * 2.0 ** -39
        tiny = half_step * float(args[4].double().norm() ** 2 + args[5].double().norm() ** 2) ** 0.5
        dx = tg.gated_backward(*args)[0]
        for r in range(rows):
            row = want["dx"][r]
            assert far(dx[r], row) <= 2.0 ** -11 + tiny / float(row.norm()), (r, largest)


def test_not_finite():
    """An infinite or NaN gradient stays in its own row and column, and the others are scaled without it."""
    args = problem(40, 64, 72, 2e-5, 0.05, 30.0, 30.0, seed=4)
    plain = tg.gated_backward(*args)
    for bad in (float("inf"), float("nan")):
        dh = args[0].clone()
        dh[3, 5] = bad
        dx, dwg, dwu = tg.gated_backward(dh, *args[1:])
        keep = torch.arange(40, device="cuda") != 3
        assert torch.equal(dx[keep], plain[0][keep]) and not torch.isfinite(dx[3]).any()
        cols = torch.arange(72, device="cuda") != 5
        want = exact(args[0], *args[1:], "silu")[0]
        for got, name in ((dwg, "dwg"), (dwu, "dwu")):
            assert torch.isfinite(got[:, cols]).all() and not torch.isfinite(got[:, 5]).any()
            assert far(got[:, cols], want[name][:, cols]) <= 2.0 ** -11


def test_nothing_and_graphs():
    """No gradient at all, and a captured call whose inputs change by more than the range."""
    args = problem(70, 136, 200, 0.0, 1.0, 1.0, 1.0)
    for t in tg.gated_backward(*args):
        assert not t.any()
    dh = args[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tg.gated_backward(*args)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = tg.gated_backward(*args)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for size in (1e-5, 1.0, 3e3, 1e-3):
        dh.copy_(torch.randn(dh.shape, generator=gen, device="cuda") * size)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, tg.gated_backward(*args)))
