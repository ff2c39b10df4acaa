"""Targets and gradients of losses that do not lie next to each other: what autograd and data loaders hand over."""

import pytest
import torch

import persistent_warp_specialized_gb300 as tg
from gpu_helpers import ensure_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    ensure_library()


@pytest.mark.parametrize("rows", [1, 7, 70])
def test_strided_rows(rows):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((rows, 136), generator=gen, device="cuda").bfloat16()
    w = torch.randn((777, 136), generator=gen, device="cuda").bfloat16() / 8
    tokens = torch.randint(0, 777, (rows, 3), generator=gen, device="cuda")
    both = torch.rand((rows, 2), generator=gen, device="cuda")
    targets = tokens[:, 1]
    loss, lse = tg.linear_cross_entropy(x, w, targets)
    want = tg.linear_cross_entropy(x, w, targets.clone())
    assert torch.equal(loss, want[0]) and torch.equal(lse, want[1])
    spread = torch.stack([lse, lse], dim=1)[:, 1]
    for dloss in (both[:, 0], torch.ones((), device="cuda").expand(rows), both[:, 1].flip(0)):
        got = tg.linear_cross_entropy_backward(dloss, x, w, targets, spread)
        want = tg.linear_cross_entropy_backward(dloss.clone(memory_format=torch.contiguous_format), x, w,
                                                targets.clone(), lse)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_gradient_that_autograd_hands_over():
    """As the backward pass of an autograd function calls it, on a stream of its own and in a graph too."""

    class Loss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, targets):
            loss, lse = tg.linear_cross_entropy(x, w, targets)
            ctx.save_for_backward(x, w, targets, lse)
            return loss

        @staticmethod
        def backward(ctx, dloss):
            assert not dloss.is_contiguous()
            x, w, targets, lse = ctx.saved_tensors
            return tg.linear_cross_entropy_backward(dloss, x, w, targets, lse) + (None,)

    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((33, 64), generator=gen, device="cuda").half().requires_grad_()
    w = (torch.randn((321, 64), generator=gen, device="cuda") / 8).half().requires_grad_()
    targets = torch.randint(0, 321, (33,), generator=gen, device="cuda")
    grads = torch.autograd.grad(Loss.apply(x, w, targets).sum(), (x, w))
    _, lse = tg.linear_cross_entropy(x.detach(), w.detach(), targets)
    want = tg.linear_cross_entropy_backward(torch.ones(33, device="cuda"), x.detach(), w.detach(), targets, lse)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    dloss = torch.full((1,), 0.5, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    args = x.detach(), w.detach(), targets, lse
    with torch.cuda.stream(side):
        tg.linear_cross_entropy_backward(dloss.expand(33), *args)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = tg.linear_cross_entropy_backward(dloss.expand(33), *args)
    dloss.fill_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
