"""The fused products on integers, whose sums are exact in fp32 whatever their order: every result is the exact
sum, rounded once.  A product that is left out or counted twice shows in it, however long the sum.

Products are of integers in [-2, 2], K goes up to 174230, so a sum is below 2^24.  Which way through the
kernels each size takes is held fast in tests/test_fused_ways_host.py: clusters and groups of them, split
sums, several segments, halves of tiles, two matrices along K or N, pieces of a vocabulary.
"""

import pytest
import torch

import fused_ref as ref
import persistent_warp_specialized_gb300 as tg
from fused_exact_sizes import GATED_BWD, GATED_FWD, INPUT_GRADS, XENT_BWD, XENT_FWD
from gpu_helpers import ensure_library

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def library():
    ensure_library()


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(shape, dtype, gen, most=2):
    return torch.randint(-most, most + 1, shape, generator=gen, device="cuda").to(dtype)


def same(got, want, what):
    """got is want, which fp32 holds exactly, rounded to got's type."""
    assert torch.equal(want.float().to(F64), want), "the sums are not exact in fp32"
    torch.cuda.synchronize()
    assert tg.tg_device_status() == 0
    bad = got != want.to(got.dtype)
    if bad.any():
        at = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} differ; first at {at}: "
                             f"{got[tuple(at)].item()}, not {want[tuple(at)].item()}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,outs", INPUT_GRADS)
def test_input_grad(rows, cols, outs, dtype):
    gen, dt = generator(1), TYPES[dtype]
    dy, w = ints((rows, outs), dt, gen), ints((cols, outs), dt, gen)
    same(tg.input_grad(dy, w), dy.to(F64) @ w.to(F64).t(), "dx")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,outs", GATED_FWD)
def test_gated_forward(rows, cols, outs, dtype):
    gen, dt = generator(2), TYPES[dtype]
    x = ints((rows, cols), dt, gen)
    wg, wu = ints((cols, outs), dt, gen) / 16, ints((cols, outs), dt, gen) / 16
    h, g, u = tg.gated_forward(x, wg, wu, keep=True)
    g64, u64 = x.to(F64) @ wg.to(F64), x.to(F64) @ wu.to(F64)
    same(g, g64, "g")
    same(u, u64, "u")
    want = (ref.gate(g64, "silu")[0] * u64).cpu()
    # as fused_ref.gated, with g and u exact
    ref.assert_within(h, want, ref.rounding(want, dt) + ref.FUNCTION * want.abs(), "h")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,outs", GATED_BWD)
def test_gated_backward(rows, cols, outs, dtype, act):
    """act is 32 and its derivative 1 at g = 32, both are 0 at -200; so dg = dh u and du = 32 dh, or 0."""
    gen, dt = generator(3), TYPES[dtype]
    x, wg, wu = ints((rows, cols), dt, gen), ints((cols, outs), dt, gen), ints((cols, outs), dt, gen)
    dh = ints((rows, outs), dt, gen, 1) / 32
    u = ints((rows, outs), dt, gen, 1) * 32
    on = torch.rand((rows, outs), generator=gen, device="cuda") < 0.7
    g = torch.where(on, 32.0, -200.0).to(dt)
    dx, dwg, dwu = tg.gated_backward(dh, g, u, x, wg, wu, act=act)
    dg, du = (dh.to(F64) * u.to(F64) * on), dh.to(F64) * 32 * on
    same(dx, dg @ wg.to(F64).t() + du @ wu.to(F64).t(), "dx")
    same(dwg, x.to(F64).t() @ dg, "dwg")
    same(dwu, x.to(F64).t() @ du, "dwu")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,vocab", XENT_FWD)
def test_loss(rows, cols, vocab, dtype):
    """Every row has one word that is far ahead of all others: lse is its logit, and the loss the difference
    between that and the target's."""
    gen, dt = generator(4), TYPES[dtype]
    base = max(1, min(rows, vocab // 2))
    kinds = ints((base, cols), dt, gen)
    x = kinds[torch.arange(rows, device="cuda") % base]
    w = ints((vocab, cols), dt, gen)
    ahead = torch.randperm(vocab, generator=gen, device="cuda")[:base]
    w[ahead] = kinds
    targets = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    targets[-1] = vocab - 1
    logits = x.to(F64) @ w.to(F64).t()
    top = logits.max(dim=1).values
    if vocab > 1:      # e^-104 is nothing beside 1 in fp32, nor are 2^16 of them
        assert (logits.sort(dim=1).values[:, -2] < top - 120).all()
    loss, lse = tg.linear_cross_entropy(x, w, targets)
    same(lse, top, "lse")
    same(loss, top - logits.gather(1, targets[:, None])[:, 0], "loss")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,vocab", XENT_BWD)
def test_loss_gradients(rows, cols, vocab, dtype):
    """Logits of 0 and -96 under an lse of 0 are probabilities of exactly 1 and 0.  The first 8 columns make the
    logits; of the others half are in x alone and half in w alone, so that they show in dw and in dx."""
    gen, dt = generator(5), TYPES[dtype]
    x, w = ints((rows, cols), dt, gen), ints((vocab, cols), dt, gen)
    half = 8 + (cols - 8) // 2
    x[:, :8], x[:, half:], w[:, 8:half] = 0, 0, 0
    column = torch.arange(rows, device="cuda") % 8
    x[torch.arange(rows, device="cuda"), column] = 1
    out = torch.rand((vocab, 8), generator=gen, device="cuda") < 0.5
    w[:, :8] = torch.where(out, -96.0, 0.0).to(dt)
    targets = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    targets[-1] = vocab - 1
    targets[::5] = -100
    dloss = 2.0 ** torch.randint(-3, 3, (rows,), generator=gen, device="cuda").float()
    dloss *= torch.randint(0, 2, (rows,), generator=gen, device="cuda") * 2 - 1
    d = (~out).to(F64).t()[column]
    counts = targets != -100
    d[counts.nonzero()[:, 0], targets[counts]] -= 1
    d *= (dloss.to(F64) * counts)[:, None]
    want_dx, want_dw = d @ w.to(F64), d.t() @ x.to(F64)
    del d
    lse = torch.zeros(rows, device="cuda")
    n = tg.tg_xent_bwd_workspace_bytes(rows, cols, vocab)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")       # NaN in either type
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    for a, b in ((dx, dw), (dx, None), (None, dw)):
        dx.fill_(float("nan"))
        dw.fill_(float("nan"))
        tg.tg_xent_bwd(dloss, x, w, targets, lse, a, b, rows, cols, vocab, cols, cols, cols, cols, -100, dtype,
                       ws)
        if a is not None:
            same(dx, want_dx, "dx")
        if b is not None:
            same(dw, want_dw, "dw")
