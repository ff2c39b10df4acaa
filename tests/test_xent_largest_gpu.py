"""The cross entropy of the largest vocabulary, 2^31 - 1 words: places past the last tile do not fit 32 bits.
Skipped when the device lacks the memory (34 GB of weights, 17 GB of statistics)."""

import pytest
import torch

import fused_ref as ref
import persistent_warp_specialized_gb300 as tg
from gpu_helpers import ensure_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    ensure_library()


@pytest.mark.parametrize("rows", [64, 65])
def test_loss_of_2_to_31_words(rows):
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB of free device memory")
    cols, vocab, last = 8, 2 ** 31 - 1, 300
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-2, 3, (rows, cols), generator=gen, device="cuda").half()
    w = torch.zeros((vocab, cols), dtype=torch.float16, device="cuda")
    w[-last:] = torch.randint(-2, 3, (last, cols), generator=gen, device="cuda").half()
    # all of the last words are somebody's target, the very last one too
    targets = vocab - 1 - (torch.arange(rows, device="cuda") * 5) % last
    logits = x.double() @ w[-last:].double().t()
    want = torch.log((vocab - last) + torch.exp(logits).sum(dim=1))
    hit = logits.gather(1, (targets - (vocab - last))[:, None])[:, 0]
    loss, lse = tg.linear_cross_entropy(x, w, targets)
    torch.cuda.synchronize()
    assert tg.tg_device_status() == 0
    # as fused_ref.xent, with exact logits; the sum is of 2^31 ones, whose partial sums are multiples of 64
    bound = 2 * ref.FUNCTION + 2.0 ** -22 * want.abs()
    ref.assert_within(lse, want.cpu(), bound.cpu(), "lse")
    ref.assert_within(loss, (want - hit).cpu(), (bound + 2.0 ** -22 * hit.abs()).cpu(), "loss")
