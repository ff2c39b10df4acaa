"""How exact the cross entropy is where fp32 sums decide: lse of long sums in norm, and the gradients of rows whose
target is nearly certain."""

import pytest
import torch

import persistent_warp_specialized_gb300 as tg
from gpu_helpers import ensure_library

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def library():
    ensure_library()


def done():
    torch.cuda.synchronize()
    assert tg.tg_device_status() == 0


# few rows, in clusters and alone; whole tiles; logits from split sums
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,vocab", [(16, 8192, 4000), (64, 8192, 20000), (65, 4096, 20000), (300, 8192, 20000),
                                             (100, 8192, 259), (155, 4432, 1961)])
def test_long_sums(rows, cols, vocab, dtype):
    """The tensor core truncates as it adds.  A segment of at most 512 products takes 32 steps of 16, each of which
    loses less than a unit, 2^-23 of the sum so far: half of that, of half the sum, on average, so 2^-20 of
    the sum (products of one sign, which these are not, lose up to twice as much).  Over 4096 products without
    a new accumulator it would be eight times as much.  Everything else, the exponentials, the logarithm and its
    rounding, is below 2^-22 of an lse of 8 or more."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((rows, cols), generator=gen, device="cuda").to(TYPES[dtype])
    w = (torch.randn((vocab, cols), generator=gen, device="cuda") * 4 * cols ** -0.5).to(TYPES[dtype])
    targets = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    loss, lse = tg.linear_cross_entropy(x, w, targets)
    done()
    logits = x.double() @ w.double().t()
    want = torch.logsumexp(logits, dim=1)
    assert want.min() > 8
    assert (lse - want).norm() <= (2 ** -20 + 2 ** -22) * want.norm()
    hit = logits.gather(1, targets[:, None])[:, 0]
    # a target's logit is as much off, of its own size
    assert (loss - (want - hit)).norm() <= (2 ** -20 + 2 ** -22) * (want.norm() + hit.norm())


# few rows up to the last; the pair kernel from the first; logits from split sums
@pytest.mark.parametrize("rows,cols,vocab", [(5, 4096, 2000), (16, 4096, 2000), (33, 4096, 2000), (64, 4096, 2000),
                                             (65, 4096, 20001), (300, 4096, 10007), (100, 8192, 259)])
def test_gradients_of_nearly_certain_targets(rows, cols, vocab):
    """With 1 - p = 2^-11 an error of p counts 2^11 times.  The backward pass makes a row's logits as the forward
    pass made them, so in p = exp(l - lse) what the tensor core truncated cancels.  What remains: half a step of
    lse (below 16: 2^-21), the exponential (2^-22) and p's own rounding, below 2^-20 in all, 2^-9 of 1 - p.
    Gradients of logits and the results are rounded besides, 2^-11 each, results below 2^-14 by half of fp16's
    smallest step, 2^-25: many are, with 1 - p of 2^-11 and weights of 2^-2 to 2^-7."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((rows, cols), generator=gen, device="cuda").half()
    w = (torch.randn((vocab, cols), generator=gen, device="cuda") * cols ** -0.5).half()
    targets = torch.randperm(vocab, generator=gen, device="cuda")[:rows]
    # the sum of the other words' exponentials is about vocab e^(1/2)
    ahead = torch.log(torch.tensor(vocab * 2.0 ** 11)) + 0.5
    w[targets] = (x.double() * (ahead / (x.double() ** 2).sum(dim=1, keepdim=True))).half()
    logits = x.double() @ w.double().t()
    want = torch.logsumexp(logits, dim=1)
    assert want.max() < 32
    d = torch.exp(logits - want[:, None])
    at = torch.arange(rows, device="cuda")
    d[at, targets] = torch.expm1(logits[at, targets] - want)      # p - 1
    short = d[at, targets].neg()
    assert (short > 2.0 ** -13).all() and (short < 2.0 ** -9).all()
    _, lse = tg.linear_cross_entropy(x, w, targets)
    dx, _ = tg.linear_cross_entropy_backward(torch.ones(rows, device="cuda"), x, w, targets, lse)
    done()
    error = (dx - d @ w.double()).norm(dim=1)
    of = (d.abs() @ w.double().abs()).norm(dim=1)
    step = torch.where(want < 16, 2.0 ** -20, 2.0 ** -19)      # of lse's half step and the rest
    bound = (step / short + 2 * 2.0 ** -11) * of + 2.0 ** -25 * cols ** 0.5
    assert (error <= bound).all(), float((error / bound).max())
