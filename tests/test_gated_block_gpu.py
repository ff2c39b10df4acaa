"""Norm, gated projections, down projection and cross entropy as a training step runs them together: the
example runs, and its gradients are those of the whole formula."""

import os
import sys

import pytest
import torch

import persistent_warp_specialized_gb300 as tg
from gpu_helpers import ensure_library

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    ensure_library()
    import gated_block_step

    return gated_block_step


def test_it_runs(example):
    losses = example.main(["--rows", "96", "--cols", "64", "--outs", "136", "--vocab", "301", "--steps", "3"])
    assert len(losses) == 3 and all(0 < v < 100 for v in losses)
    assert tg.tg_device_status() == 0


# few rows, and more than a pair's tile; an odd vocabulary
@pytest.mark.parametrize("rows,cols,outs,vocab", [(5, 64, 72, 131), (40, 96, 264, 1003), (300, 128, 392, 515)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_gradients(example, rows, cols, outs, vocab, dtype):
    block = example.GatedBlock(cols, outs, vocab, dtype, seed=3)
    for name in ("wg", "wu", "wd", "e"):
        block.p[name] = block.half(name).float()      # so that the formula has the same weights
    gen = torch.Generator().manual_seed(4)
    x = torch.randn((rows, cols), generator=gen).to(dtype).cuda()
    targets = torch.randint(0, vocab, (rows,), generator=gen).cuda()
    targets[::6] = -100
    dloss = torch.rand(rows, generator=gen).cuda()
    loss, saved = block.forward(x, targets)
    got = block.backward(dloss, saved)
    torch.cuda.synchronize()
    assert tg.tg_device_status() == 0

    f = torch.nn.functional
    p = {k: v.double().requires_grad_() for k, v in block.p.items()}
    xd = x.double().requires_grad_()
    y = f.layer_norm(xd, (cols,), p["gamma"], p["beta"], 1e-5)
    z = xd + (f.silu(y @ p["wg"]) * (y @ p["wu"])) @ p["wd"]
    want = f.cross_entropy(z @ p["e"].t(), targets, reduction="none", ignore_index=-100)
    (want * dloss.double()).sum().backward()
    # Roundings on the way to a gradient: y, g and u, h, h Wd, z, dl, dz, dh, dg and du, dy, the result; 11,
    # each of at most eps / 2 of its matrix in norm.  A relative error of a matrix reaches the gradients up to
    # about four times as large here (two factors of a product, act' beside act, values that cancel against
    # the residual).  Wd's gradient has h in 8 bits besides: E4M3 is off by up to 2^-4 in a value (an eighth for
    # a block's largest), 2^-5 in norm.
    bound = 11 * 4 * torch.finfo(dtype).eps / 2
    far = {k: float((got[k].double() - t.grad).norm() / t.grad.norm()) for k, t in list(p.items()) + [("x", xd)]}
    far["loss"] = float((loss.double() - want).detach().norm() / want.detach().norm())
    for name, d in far.items():
        assert d <= bound + (2 ** -5 if name == "wd" else 0), (name, far)


def test_two_threads_at_once():
    """Two host threads, each on a stream of its own, get what one alone gets: calls share no scratch."""
    import threading

    gen = torch.Generator(device="cuda").manual_seed(5)

    def matrix(rows, cols, scale=1.0):
        return (torch.randn((rows, cols), generator=gen, device="cuda") * scale).bfloat16()

    sets = [(matrix(r, 264), matrix(264, 520, 0.06), matrix(264, 520, 0.06), matrix(3001, 264, 0.06),
             torch.randint(0, 3001, (r,), generator=gen, device="cuda")) for r in (5, 300)]

    def step(x, wg, wu, e, targets):
        h, g, u = tg.gated_forward(x, wg, wu, keep=True)
        loss, lse = tg.linear_cross_entropy(x, e, targets)
        return (h, loss, lse, tg.input_grad(h, wg)) + tuple(tg.gated_backward(h, g, u, x, wg, wu)) + tuple(
            tg.linear_cross_entropy_backward(torch.ones_like(loss), x, e, targets, lse))

    alone = [step(*s) for s in sets]
    torch.cuda.synchronize()
    got, raised = [[], []], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[i].append(step(*sets[i]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # the main thread fails the test
            raised.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not raised and tg.tg_device_status() == 0
    for i in range(2):
        assert len(got[i]) == 20
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(alone[i], outs))
