"""The input gradient and the gated projections, forward and backward, against 64 bits (tests/fused_ref.py
has the bounds)."""

import pytest
import torch

import fused_ref as ref
import persistent_warp_specialized_gb300 as tg
from gpu_helpers import ensure_library

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def library():
    ensure_library()


def normal(shape, dtype, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def ints(shape, dtype, seed, most=2):
    gen = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=gen).to(dtype)


def check(got, want, what=""):
    torch.cuda.synchronize()
    assert tg.tg_device_status() == 0
    for name, (value, bound) in want.items():
        ref.assert_within(got[name], value, bound, f"{what} {name}")


# rows, cols, outs: one token; edges of warps (32), CTAs (128), pairs (256), atoms (64) and k-blocks (128);
# K split into ranges (few tiles, long K); several segments of 1024; half-width units (77 tiles and more).
# Up to 64 rows: 16, 32 or 64 to an MMA, tiles of 128, clusters that share a tile, groups of them (17, 300, 20000)
GRADS = [(1, 8, 8), (3, 136, 72), (33, 128, 128), (129, 264, 200), (255, 520, 1032), (257, 256, 2048),
         (2, 2048, 4104), (64, 640, 3000), (17, 304, 20000), (16, 20000, 72), (300, 392, 8192),
         (1300, 3200, 256), (2600, 2600, 136)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,outs", GRADS)
def test_input_grad(rows, cols, outs, dtype):
    dt = TYPES[dtype]
    dy, w = normal((rows, outs), dt, 1), normal((cols, outs), dt, 2, outs ** -0.5)
    dx, s = ref.product(dy, w.t())
    got = tg.input_grad(dy.cuda(), w.cuda())
    check({"dx": got}, {"dx": (dx, ref.rounding(dx, dt) + 1.01 * ref.gamma(outs) * s)})


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,outs", [(77, 200, 64), (257, 300 * 8, 56), (1, 640, 8), (700, 1288, 16)])
def test_input_grad_of_integers_is_exact(rows, cols, outs, dtype):
    dt = TYPES[dtype]
    dy, w = ints((rows, outs), dt, 3), ints((cols, outs), dt, 4)     # sums of at most 64 * 4
    got = tg.input_grad(dy.cuda(), w.cuda()).cpu()
    assert torch.equal(got.double(), dy.double() @ w.double().t())


# rows, cols, outs of the gated projections; outs 128 wide tiles, half units 64
LAYERS = [(1, 8, 8), (1, 1024, 2048), (2, 136, 72), (5, 2056, 1000), (8, 600, 264), (9, 520, 304), (33, 128, 128),
          (64, 344, 200), (129, 264, 200),
          (200, 1024, 640), (257, 72, 1032), (1300, 136, 2000), (300, 4104, 392)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,cols,outs", LAYERS)
def test_gated_forward(rows, cols, outs, act, dtype):
    dt = TYPES[dtype]
    x = normal((rows, cols), dt, 5)
    wg, wu = normal((cols, outs), dt, 6, 2 * cols ** -0.5), normal((cols, outs), dt, 7, cols ** -0.5)
    want = ref.gated(x, wg, wu, act)
    args = x.cuda(), wg.cuda(), wu.cuda()
    h, g, u = tg.gated_forward(*args, act=act, keep=True)
    check({"h": h, "g": g, "u": u}, want, "kept")
    alone = tg.gated_forward(*args, act=act)
    assert torch.equal(alone, h)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,cols,outs", LAYERS)
def test_gated_backward(rows, cols, outs, act, dtype):
    dt = TYPES[dtype]
    x, dh = normal((rows, cols), dt, 8), normal((rows, outs), dt, 9, 0.1)
    wg, wu = normal((cols, outs), dt, 10, outs ** -0.5), normal((cols, outs), dt, 11, outs ** -0.5)
    g, u = normal((rows, outs), dt, 12, 1.5), normal((rows, outs), dt, 13)
    want = ref.gated_grads(dh, g, u, x, wg, wu, act)
    got = tg.gated_backward(*(t.cuda() for t in (dh, g, u, x, wg, wu)), act=act)
    check(dict(zip(("dx", "dwg", "dwu"), got)), want)


def test_gradient_is_that_of_the_forward_pass():
    # against differences of the forward formula in 64 bits
    gen = torch.Generator().manual_seed(14)
    x, wg, wu = (torch.randn(s, generator=gen).bfloat16() for s in ((3, 16), (16, 24), (16, 24)))
    wg, wu = wg / 4, wu / 4
    dh = torch.randn((3, 24), generator=gen).bfloat16()
    for act in ("silu", "gelu"):
        g, u = (x.double() @ wg.double()).bfloat16(), (x.double() @ wu.double()).bfloat16()
        got = [t.double().cpu() for t in tg.gated_backward(
            *(t.cuda() for t in (dh, g, u, x, wg, wu)), act=act)]

        def value(x, wg, wu):
            return (ref.gate(x @ wg, act)[0] * (x @ wu) * dh.double()).sum()

        base = [x.double(), wg.double(), wu.double()]
        for i, name in enumerate(("dx", "dwg", "dwu")):
            step = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)
            ahead, behind = list(base), list(base)
            ahead[i], behind[i] = base[i] + 1e-5 * step, base[i] - 1e-5 * step
            slope = (value(*ahead) - value(*behind)) / 2e-5
            # g, u, dg, du and the result rounded to 8 bits: 2^-8 each, of the sum of magnitudes
            assert abs((got[i] * step).sum() - slope) <= 5 * 2 ** -8 * (got[i] * step).abs().sum(), name


def test_column_slices_and_guards():
    """Weights side by side in one matrix, inputs and outputs inside wider ones; what lies around the
    outputs stays as it was."""
    dt, rows, cols, outs = torch.bfloat16, 70, 136, 200
    both = normal((cols, 2 * outs), dt, 15, 0.1).cuda()
    wide = normal((rows + 4, cols + 24), dt, 16).cuda()
    x, wg, wu = wide[2:2 + rows, 8:8 + cols], both[:, :outs], both[:, outs:]
    buf = torch.full((rows + 8, outs + 16), 7.0, dtype=dt, device="cuda")
    h = tg.gated_forward(x, wg, wu, out=buf[4:4 + rows, 8:8 + outs])
    check({"h": h}, {"h": ref.gated(x.cpu(), wg.cpu(), wu.cpu(), "silu")["h"]})
    buf[4:4 + rows, 8:8 + outs] = 7.0
    assert (buf == 7.0).all()
    dy = normal((rows, 2 * outs), dt, 17).cuda()[:, outs:]
    gbuf = torch.full((rows + 3, cols + 8), 7.0, dtype=dt, device="cuda")
    dx = tg.input_grad(dy, wu, out=gbuf[:rows, 8:])
    want, s = ref.product(dy.cpu(), wu.cpu().t())
    check({"dx": dx}, {"dx": (want, ref.rounding(want, dt) + 1.01 * ref.gamma(outs) * s)})
    gbuf[:rows, 8:] = 7.0
    assert (gbuf == 7.0).all()


@pytest.mark.parametrize("rows,ld", [(40, 1 << 27), (600, 1 << 23)])
def test_results_more_than_2_to_32_values_apart(rows, ld):
    """Row strides that take the last rows' offsets past 32 bits, of inputs and outputs."""
    dt, cols, outs = torch.float16, 136, 72
    wide = torch.empty((rows, ld), dtype=dt, device="cuda")
    x, h = wide[:, 64:64 + cols], wide[:, 1024:1024 + outs]
    x.copy_(normal((rows, cols), dt, 30))
    wg, wu = normal((cols, outs), dt, 31, 0.1).cuda(), normal((cols, outs), dt, 32, 0.1).cuda()
    tg.gated_forward(x, wg, wu, out=h)
    same = tg.gated_forward(x.contiguous(), wg, wu)
    dx = tg.input_grad(h, wg, out=wide[:, 2048:2048 + cols])
    torch.cuda.synchronize()
    assert torch.equal(h, same) and torch.equal(dx, tg.input_grad(same, wg))
    n = tg.tg_gated_bwd_workspace_bytes(rows, cols, outs)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dwg, dwu = torch.empty_like(wg), torch.empty_like(wu)
    back = wide[:, 4096:4096 + cols]
    tg.tg_gated_bwd(h, h, h, x, wg, wu, back, dwg, dwu, rows, cols, outs, ld, ld, ld, ld, outs, outs, ld, outs,
                    outs, "silu", "f16", ws)
    want = tg.gated_backward(same, same, same, x.contiguous(), wg, wu)
    assert all(torch.equal(a, b) for a, b in zip((back, dwg, dwu), want))


def raw_bwd(dh, g, u, x, wg, wu, dx, dwg, dwu, act="silu"):
    rows, outs, cols = dh.shape[0], dh.shape[1], wg.shape[0]
    n = tg.tg_gated_bwd_workspace_bytes(rows, cols, outs)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    tg.tg_gated_bwd(dh, g, u, x, wg, wu, dx, dwg, dwu, rows, cols, outs, outs, outs, outs, cols, outs, outs,
                    cols, outs, outs, act, "f16", ws)


def test_gradients_asked_for_one_by_one_and_empty_sizes():
    dt = torch.float16
    rows, cols, outs = 40, 64, 72
    dh, g, u = (normal((rows, outs), dt, s).cuda() for s in (18, 19, 20))
    x = normal((rows, cols), dt, 21).cuda()
    wg, wu = normal((cols, outs), dt, 22).cuda(), normal((cols, outs), dt, 23).cuda()
    all_ = tg.gated_backward(dh, g, u, x, wg, wu)
    dx, dwg, dwu = torch.empty_like(all_[0]), torch.empty_like(all_[1]), torch.empty_like(all_[2])
    raw_bwd(dh, g, u, None, wg, wu, dx, None, None)
    raw_bwd(dh, g, u, x, wg, wu, None, dwg, dwu)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(all_, (dx, dwg, dwu)))
    # no rows: gradients of weights are zero; no columns of h: so is dx
    assert not tg.gated_forward(torch.empty((rows, 0), dtype=dt, device="cuda"), wg[:0], wu[:0]).any()
    zero = tg.gated_backward(dh[:0], g[:0], u[:0], x[:0], wg, wu)
    assert zero[0].shape == (0, cols) and not zero[1].any() and not zero[2].any()
    none = tg.gated_backward(dh[:, :0], g[:, :0], u[:, :0], x, wg[:, :0], wu[:, :0])
    assert none[0].shape == (rows, cols) and not none[0].any()
    assert not tg.gated_forward(x[:, :0], wg[:0], wu[:0]).any()
    assert not tg.input_grad(dh[:, :0], wg[:, :0]).any()
    assert tg.input_grad(dh[:0], wg).shape == (0, cols)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", TYPES)
def test_extreme_gates(act, dtype):
    """Gates of any size: act is 0 or g far out, its derivative 0 or 1, and NaN stays in its own row."""
    dt = TYPES[dtype]
    top = torch.finfo(dt).max
    vals = torch.tensor([0.0, -0.0, 5e-8, -5e-8, 1.0, -1.0, 9.0, -9.0, 15.9, -15.9, 16.1, -16.1, 40.0, -40.0,
                         88.0, -88.0, 90.0, -90.0, 104.0, -104.0, 1e4, -1e4, top, -top],
                        dtype=torch.float64).to(dt)
    outs = vals.numel()
    # x = (1, 0, ...), so that g is Wg's first row
    x = torch.zeros((2, 8), dtype=dt)
    x[0, 0] = 1
    x[1, 1] = float("nan")
    wg, wu = torch.zeros((8, outs), dtype=dt), torch.zeros((8, outs), dtype=dt)
    wg[0], wu[0] = vals, 1.0
    h, g, u = (t.cpu() for t in tg.gated_forward(x.cuda(), wg.cuda(), wu.cuda(), act=act, keep=True))
    assert torch.equal(g[0], vals) and (u[0] == 1).all() and torch.isnan(h[1]).all()
    a, slope = ref.gate(vals.double().clamp(-200, 200), act)
    a = torch.where(vals.double().abs() > 200, vals.double().clamp(min=0), a)
    ref.assert_within(h[0], a, ref.rounding(a, dt) + 2 * ref.FUNCTION * a.abs() + 1e-35, "h")
    one = torch.ones((2, outs), dtype=dt)
    dx, dwg, dwu = tg.gated_backward(one.cuda(), torch.stack([vals, vals]).cuda(), one.cuda(),
                                     torch.nan_to_num(x).cuda(), wg.cuda(), wu.cuda(), act=act)
    assert torch.isfinite(dwg).all()
    ref.assert_within(dwg[0], slope, 2 * ref.rounding(slope, dt) + 8 * ref.FUNCTION, "act'")


def test_equal_calls_give_equal_bits_on_any_stream_and_in_graphs():
    dt, rows, cols, outs = torch.bfloat16, 40, 2048, 520       # K is split: workspaces and joins
    x, dh = normal((rows, cols), dt, 24).cuda(), normal((rows, outs), dt, 25).cuda()
    wg, wu = normal((cols, outs), dt, 26, 0.02).cuda(), normal((cols, outs), dt, 27, 0.02).cuda()

    def run():
        h, g, u = tg.gated_forward(x, wg, wu, keep=True)
        return (h, g, u) + tuple(tg.gated_backward(dh, g, u, x, wg, wu)) + (tg.input_grad(dh, wg),)

    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        graphs, outs_ = [], []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                outs_.append(run())
            graphs.append(graph)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(3):                       # two graphs at once, each with workspaces of its own
        with torch.cuda.stream(side):
            graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert tg.tg_device_status() == 0
    for got in outs_ + [run()]:
        assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.parametrize("rows,cols,outs,ctas", [
    (512, 512, 1024, (0, 1)),       # the even and the odd CTA of pair 0
    (20, 512, 2048, (0, 5)),        # few rows: the first and a later CTA of a cluster
    (20, 25000, 512, (3,))])        # and one without a cluster
def test_the_watchdog_stops_a_missing_fill(rows, cols, outs, ctas):
    dt = torch.bfloat16
    dy, w = normal((rows, outs), dt, 28).cuda(), normal((cols, outs), dt, 29).cuda()
    dx = torch.empty((rows, cols), dtype=dt, device="cuda")
    n = tg.tg_input_grad_workspace_bytes(rows, cols, outs)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    args = (dy, w, dx, rows, cols, outs, outs, outs, cols, "bf16", ws)
    for cta in ctas:
        with pytest.raises(tg.TgError) as e:
            tg.tg_input_grad_debug(*args, watchdog_ns=20_000_000, inject_skip_phase=(cta << 32) + 1)
        assert e.value.code == tg.TG_ERR_TIMEOUT
    assert tg.tg_input_grad_debug(*args) == 0
    assert torch.equal(dx, tg.input_grad(dy, w))


def test_refusals_that_need_a_device():
    x = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((64, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(tg.TgError, match="overlaps"):
        tg.input_grad(x, w, out=x)
    with pytest.raises(tg.TgError, match="overlaps"):
        tg.gated_forward(x, w, w, out=w[:8])
    with pytest.raises(tg.TgError, match="workspace"):
        tg.tg_gated_bwd(x, x, x, x, w, w, torch.empty_like(x), None, None, 8, 64, 64, *[64] * 9, "silu",
                        "bf16")
    with pytest.raises(tg.TgError, match="device memory"):
        tg.input_grad(x.cpu().pin_memory(), w, out=torch.empty_like(x))
