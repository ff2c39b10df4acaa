"""The cross entropy of a vocabulary projection and its gradients, against 64 bits (tests/fused_ref.py has the
bounds)."""

import pytest
import torch

import fused_ref as ref
import persistent_warp_specialized_gb300 as tg
from gpu_helpers import ensure_library

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
IGNORE = -100


@pytest.fixture(scope="module", autouse=True)
def library():
    ensure_library()


def problem(rows, cols, vocab, dtype, seed, ignored=0.2):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=gen).to(dtype)
    w = (torch.randn((vocab, cols), generator=gen) * 2 * cols ** -0.5).to(dtype)
    targets = torch.randint(0, vocab, (rows,), generator=gen)
    targets[torch.rand(rows, generator=gen) < ignored] = IGNORE
    return x, w, targets


def done():
    torch.cuda.synchronize()
    assert tg.tg_device_status() == 0


# one row, one word; edges of warps, CTAs, tiles and 64-word slots; a last tile in two half units; sums of
# logits that are split (few tiles, many columns), of an odd vocabulary too; 8 of
# K, and several segments of 1024
SIZES = [(1, 8, 1), (1, 64, 500), (5, 8, 63), (33, 128, 65), (128, 264, 256), (129, 136, 257),
         (300, 2056, 1000), (155, 4432, 1961), (100, 8192, 259), (257, 64, 10007), (2600, 72, 2111)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,vocab", SIZES)
def test_loss(rows, cols, vocab, dtype):
    x, w, targets = problem(rows, cols, vocab, TYPES[dtype], 1)
    want = ref.xent(x, w, targets, IGNORE)
    loss, lse = tg.linear_cross_entropy(x.cuda(), w.cuda(), targets.cuda())
    done()
    ref.assert_within(loss, *want["loss"], "loss")
    ref.assert_within(lse, *want["lse"], "lse")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,vocab", SIZES)
def test_gradients(rows, cols, vocab, dtype):
    x, w, targets = problem(rows, cols, vocab, TYPES[dtype], 2)
    lse = ref.xent(x, w, targets, IGNORE)["lse"][0].float()
    dloss = torch.rand(rows, generator=torch.Generator().manual_seed(3)) / rows - 0.2 / rows
    want = ref.xent_grads(dloss, x, w, targets, lse, IGNORE)
    dx, dw = tg.linear_cross_entropy_backward(dloss.cuda(), x.cuda(), w.cuda(), targets.cuda(), lse.cuda())
    done()
    ref.assert_within(dx, *want["dx"], "dx")
    ref.assert_within(dw, *want["dw"], "dw")
    assert not dx.cpu()[targets == IGNORE].any()


def test_gradient_is_that_of_the_loss():
    gen = torch.Generator().manual_seed(4)
    x, w, targets = problem(6, 16, 37, torch.bfloat16, 5)
    dloss = torch.rand(6, generator=gen)
    _, lse = tg.linear_cross_entropy(x.cuda(), w.cuda(), targets.cuda())
    got = [t.double().cpu() for t in tg.linear_cross_entropy_backward(
        dloss.cuda(), x.cuda(), w.cuda(), targets.cuda(), lse)]

    def value(x, w):
        return (torch.nn.functional.cross_entropy(x @ w.t(), targets, reduction="none",
                                                  ignore_index=IGNORE) * dloss).sum()

    base = [x.double(), w.double()]
    for i in range(2):
        step = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)
        ahead, behind = list(base), list(base)
        ahead[i], behind[i] = base[i] + 1e-5 * step, base[i] - 1e-5 * step
        slope = (value(*ahead) - value(*behind)) / 2e-5
        # the gradients of the logits and the results are rounded: 2^-9 each, with room for cancellation
        assert abs((got[i] * step).sum() - slope) <= 4 * 2 ** -8 * (got[i] * step).abs().sum()


@pytest.mark.parametrize("dtype", TYPES)
def test_pieces_of_the_vocabulary(dtype):
    """More rows than one piece of 256 MiB of gradients holds: three pieces, the last one narrow."""
    rows, cols, vocab = 40000, 16, 8000
    per = (256 << 20) // (2 * rows) // 256 * 256
    assert 2 * per < vocab < 3 * per
    gen = torch.Generator(device="cuda").manual_seed(6)
    dt = TYPES[dtype]
    x = torch.randn((rows, cols), generator=gen, device="cuda").to(dt)
    w = (torch.randn((vocab, cols), generator=gen, device="cuda") * 0.5).to(dt)
    targets = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    targets[::7] = IGNORE
    dloss = torch.full((rows,), 1.0 / rows, device="cuda")
    loss, lse = tg.linear_cross_entropy(x, w, targets)
    dx, dw = tg.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    done()
    xd, wd = x.double(), w.double()
    dw_ref, total = torch.zeros_like(wd), 0.0
    ulp = torch.finfo(dt).eps / 2
    for r in range(0, rows, 4000):              # a block of rows at a time
        s = slice(r, r + 4000)
        logits = xd[s] @ wd.t()
        want = torch.logsumexp(logits, dim=1)
        # logits of 16 products, |l| < 40: gamma(16) 40 < 2^-13; then as fused_ref.xent
        assert (lse[s].double() - want).abs().max() < 2.0 ** -13 + 2 * ref.FUNCTION
        d = torch.exp(logits - want[:, None])
        keep = targets[s] != IGNORE
        rows_ = torch.arange(len(keep), device="cuda")[keep]
        d[rows_, targets[s][keep]] -= 1.0
        d *= keep[:, None] / rows
        dw_ref += d.t() @ xd[s]
        dx_ref = d @ wd
        # dl off by a rounding and by what lse and the logits are off (2^-12), of the magnitudes; the
        # result by a rounding (fp16: of a subnormal step, 2^-25)
        bound = dx_ref.abs() * ulp + (ulp + 2.0 ** -12) * 1.05 * (d.abs() @ wd.abs()) + 2.0 ** -25
        assert ((dx[s].double() - dx_ref).abs() <= bound).all()
        total = total + d.abs().t() @ xd[s].abs()
    # and fp32 sums over 40000 tokens, in segments
    bound = dw_ref.abs() * ulp + (ulp + 2.0 ** -12 + ref.gamma(2048)) * 1.05 * total + 2.0 ** -25
    assert ((dw.double() - dw_ref).abs() <= bound).all()


def test_rows_that_do_not_count_and_wrong_targets():
    x, w, targets = problem(64, 72, 300, torch.float16, 7, ignored=0.0)
    ones = torch.ones(64)
    none = torch.full_like(targets, IGNORE)
    loss, lse = tg.linear_cross_entropy(x.cuda(), w.cuda(), none.cuda())
    assert not loss.any() and torch.isfinite(lse).all()
    dx, dw = tg.linear_cross_entropy_backward(ones.cuda(), x.cuda(), w.cuda(), none.cuda(), lse)
    assert not dx.any() and not dw.any()
    # ignore_index may be a word; words past the vocabulary and below 0 are wrong, beside a tile's end too
    targets[3], targets[9], targets[20], targets[31] = 300, -1, 1 << 40, IGNORE
    targets[40] = 17
    loss, lse = (t.cpu() for t in tg.linear_cross_entropy(x.cuda(), w.cuda(), targets.cuda(),
                                                          ignore_index=17))
    wrong = torch.zeros(64, dtype=torch.bool)
    wrong[[3, 9, 20, 31]] = True
    assert torch.isnan(loss[wrong]).all() and torch.isfinite(loss[~wrong]).all()
    assert (loss[targets == 17] == 0).all() and torch.isfinite(lse).all()
    dx, dw = (t.cpu() for t in tg.linear_cross_entropy_backward(
        ones.cuda(), x.cuda(), w.cuda(), targets.cuda(), lse.cuda(), ignore_index=17))
    assert torch.isnan(dx[wrong]).all() and torch.isfinite(dx[~wrong]).all()
    assert not dx[targets == 17].any() and torch.isnan(dw).all()


def test_words_that_are_masked_out_and_special_values():
    x, w, targets = problem(40, 64, 200, torch.float16, 8, ignored=0.0)
    targets %= 100
    x[:, 0] = 1.0
    half = w.clone()
    half[100:] = 0.0
    half[100:, 0] = -65504.0                    # the type's lowest value: no probability
    got = tg.linear_cross_entropy(x.cuda(), half.cuda(), targets.cuda())
    want = ref.xent(x, w[:100], targets, IGNORE)
    for g, name in zip(got, ("loss", "lse")):
        ref.assert_within(g, *want[name], name)
    dx, dw = tg.linear_cross_entropy_backward(torch.ones(40).cuda(), x.cuda(), half.cuda(), targets.cuda(),
                                              got[1])
    grads = ref.xent_grads(torch.ones(40), x, w[:100], targets, want["lse"][0], IGNORE)
    # lse is the kernel's here, off by its bound: p by as much again
    assert not dw[100:].any()
    value, bound = grads["dw"]
    ref.assert_within(dw[:100], value, bound * 2, "dw")
    # minus infinity is no probability either; plus infinity and NaN make NaN of their rows alone
    half[100:, 0] = -float("inf")
    got = tg.linear_cross_entropy(x.cuda(), half.cuda(), targets.cuda())
    for g, name in zip(got, ("loss", "lse")):
        ref.assert_within(g, *want[name], name)
    x[5, 0], x[6, 3] = -1.0, float("nan")
    got = [t.cpu() for t in tg.linear_cross_entropy(x.cuda(), half.cuda(), targets.cuda())]
    for t in got:
        bad = torch.isnan(t)
        assert bad[5] and bad[6] and bad.sum() == 2


def test_lone_rows_of_large_and_small_weight():
    """A row's gradient is right beside rows of any other weight, down to 2^-20 of the largest."""
    for dtype in TYPES.values():
        x, w, targets = problem(4, 64, 130, dtype, 9, ignored=0.0)
        dloss = torch.tensor([1e-3, -2.0 ** -20 * 1e-3, 0.0, 1e-6])
        lse = ref.xent(x, w, targets, IGNORE)["lse"][0].float()
        want = ref.xent_grads(dloss, x, w, targets, lse, IGNORE)
        dx, dw = tg.linear_cross_entropy_backward(dloss.cuda(), x.cuda(), w.cuda(), targets.cuda(),
                                                  lse.cuda())
        ref.assert_within(dx, *want["dx"], "dx")
        ref.assert_within(dw, *want["dw"], "dw")
        for scale in (0.0, float("inf"), float("nan")):
            d = torch.full((4,), scale)
            dx, _ = tg.linear_cross_entropy_backward(d.cuda(), x.cuda(), w.cuda(), targets.cuda(),
                                                     lse.cuda())
            assert not dx.any() if scale == 0.0 else not torch.isfinite(dx).any()


def test_column_slices_streams_and_graphs():
    rows, cols, vocab = 70, 136, 777
    x, w, targets = problem(rows, cols, vocab, torch.bfloat16, 10)
    wide = torch.zeros((vocab, cols + 16), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + cols] = w.cuda()
    xs, ws, ts = x.cuda(), wide[:, 8:8 + cols], targets.cuda()
    dloss = torch.full((rows,), 1.0 / rows, device="cuda")

    def run():
        loss, lse = tg.linear_cross_entropy(xs, ws, ts)
        return (loss, lse) + tuple(tg.linear_cross_entropy_backward(dloss, xs, ws, ts, lse))

    first = run()
    whole = tg.linear_cross_entropy(xs, w.cuda(), ts)
    assert torch.equal(first[0], whole[0]) and torch.equal(first[1], whole[1])
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(side):
        run()
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                outs.append(run())
            graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(3):
        for stream, graph in ((side, graphs[0]), (other, graphs[1])):
            with torch.cuda.stream(stream):
                graph.replay()
    done()
    for got in outs + [run()]:
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_only_what_is_asked_for():
    rows, cols, vocab = 33, 64, 321
    x, w, targets = (t.cuda() for t in problem(rows, cols, vocab, torch.float16, 11))
    _, lse = tg.linear_cross_entropy(x, w, targets)
    dloss = torch.rand(rows, device="cuda")
    both = tg.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    n = tg.tg_xent_bwd_workspace_bytes(rows, cols, vocab)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    for a, b in ((dx, None), (None, dw)):
        tg.tg_xent_bwd(dloss, x, w, targets, lse, a, b, rows, cols, vocab, cols, cols, cols, cols, IGNORE,
                       "f16", ws)
    done()
    assert torch.equal(dx, both[0]) and torch.equal(dw, both[1])
    none = tg.linear_cross_entropy_backward(dloss[:0], x[:0], w, targets[:0], lse[:0])
    assert none[0].shape == (0, cols) and not none[1].any()
    with pytest.raises(tg.TgError, match="overlaps"):
        tg.tg_xent_bwd(dloss, x, w, targets, lse, x, None, rows, cols, vocab, cols, cols, cols, cols,
                       IGNORE, "f16", ws)
    with pytest.raises(tg.TgError, match="workspace"):
        tg.tg_xent_bwd(dloss, x, w, targets, lse, dx, None, rows, cols, vocab, cols, cols, cols, cols,
                       IGNORE, "f16", ws, workspace_bytes=n - 1)


@pytest.mark.parametrize("rows", [3, 70])
def test_a_vocabulary_of_more_than_2_to_31_values(rows):
    """Offsets into w and dw past 31 and 32 bits: 270000 words of 8192 columns (4.4 GB), all of them zero but
    some at the end."""
    cols, vocab, last = 8192, 270000, 7
    gen = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn((rows, cols), generator=gen, device="cuda").bfloat16()
    w = torch.zeros((vocab, cols), dtype=torch.bfloat16, device="cuda")
    w[-last:] = torch.randn((last, cols), generator=gen, device="cuda") * 0.1
    targets = torch.randint(vocab - last, vocab, (rows,), generator=gen, device="cuda")
    targets[1] = 5
    loss, lse = tg.linear_cross_entropy(x, w, targets)
    logits = x.double() @ w[-last:].double().t()
    top = logits.max(dim=1).values.clamp(min=0)
    want = top + torch.log((vocab - last) * torch.exp(-top) + torch.exp(logits - top[:, None]).sum(dim=1))
    hit = torch.zeros(rows, dtype=torch.float64, device="cuda")
    end = targets >= vocab - last
    hit[end] = logits[end].gather(1, (targets[end] - (vocab - last))[:, None])[:, 0]
    # segments of 1024 products: off by at most 2^-23 of the magnitudes each; as fused_ref.xent otherwise
    off = ref.gamma(cols) * (x.double().abs() @ w[-last:].double().abs().t()).max() + 2 * ref.FUNCTION \
        + 2.0 ** -21 * want.abs().max()
    assert (lse - want).abs().max() <= off and (loss - (want - hit)).abs().max() <= 2 * off
    dloss = torch.ones(rows, device="cuda")
    dx, dw = tg.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    done()
    p = torch.exp(logits - want[:, None])
    p[end] = p[end].scatter_add(1, (targets[end] - (vocab - last))[:, None],
                                -torch.ones_like(hit[end])[:, None])
    # p off by what lse and a logit are (2 off) and one rounding; the results by one more
    rel = 2.0 ** -8 + 3 * off
    assert (dx.double() - p @ w[-last:].double()).norm() <= 2 * rel * (p.abs() @ w[-last:].double().abs()).norm()
    got = dw[-last:].double()
    assert (got - p.t() @ x.double()).norm() <= 2 * rel * (p.abs().t() @ x.double().abs()).norm()
    d5 = -x[1].double() + torch.exp(-want) @ x.double()          # word 5: row 1's target
    assert (dw[5].double() - d5).norm() <= 2 * rel * d5.norm()
    zero = torch.exp(-want) @ x.double()                         # a word that is nobody's target
    assert (dw[vocab - last - 1].double() - zero).norm() <= 4 * rel * (torch.exp(-want) @ x.double().abs()).norm()
