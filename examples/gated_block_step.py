"""Trains one pre-norm gated feed-forward block with a residual and a vocabulary's cross entropy:

    y = layer_norm(x),  h = silu(y Wg) (y Wu),  z = x + h Wd,  loss = cross entropy of z E^T

    python examples/gated_block_step.py [--rows 2048 --cols 1024 --outs 2816 --vocab 16384 --steps 20]

No logits and no transposed weights are ever in memory: the loss and its gradients go through the
vocabulary in pieces, and what the products hand back to their inputs reads the weights as they lie.
Wd's gradient is taken from an 8-bit checkpoint of h.  Needs a GB300 and the built library (see the README).
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import persistent_warp_specialized_gb300 as tg


class GatedBlock:
    """gamma, beta [cols], Wg, Wu [cols, outs], Wd [outs, cols], E [vocab, cols]; master copies in float32."""

    def __init__(self, cols, outs, vocab, dtype, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.dtype = dtype

        def normal(*shape):
            return (torch.randn(shape, generator=gen) / cols ** 0.5).cuda()

        self.p = {"gamma": torch.ones(cols, device="cuda"), "beta": torch.zeros(cols, device="cuda"),
                  "wg": normal(cols, outs), "wu": normal(cols, outs), "wd": normal(outs, cols),
                  "e": normal(vocab, cols)}

    def half(self, name):
        return self.p[name].to(self.dtype)

    def forward(self, x, targets):
        """Each row's loss, and what the backward pass needs."""
        y, mean, rstd = tg.layer_norm(x, self.p["gamma"], self.p["beta"])
        h, g, u = tg.gated_forward(y, self.half("wg"), self.half("wu"), keep=True)
        z = x + tg.gemm(h, self.half("wd"))
        loss, lse = tg.linear_cross_entropy(z, self.half("e"), targets)
        return loss, (x, targets, mean, rstd, y, g, u, tg.ckpt8_pack(h), z, lse)

    def backward(self, dloss, saved):
        """Gradients by name, that of x among them, from the gradient of each row's loss."""
        x, targets, mean, rstd, y, g, u, kept_h, z, lse = saved
        d = {}
        dz, d["e"] = tg.linear_cross_entropy_backward(dloss, z, self.half("e"), targets, lse)
        d["wd"] = tg.ckpt8_wgrad(kept_h, dz)
        dh = tg.input_grad(dz, self.half("wd"))
        dy, d["wg"], d["wu"] = tg.gated_backward(dh, g, u, y, self.half("wg"), self.half("wu"))
        dx, d["gamma"], d["beta"] = tg.layer_norm_backward(dy, x, mean, rstd, self.p["gamma"])
        d["x"] = dz + dx
        return d


def step(block, x, targets, lr):
    """One step of gradient descent on the mean loss; returns it."""
    loss, saved = block.forward(x, targets)
    # of the sum, to keep 16-bit gradients in range
    grads = block.backward(torch.ones_like(loss), saved)
    for name, p in block.p.items():
        p -= lr / len(loss) * grads[name].float()
    return loss.mean()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=2048)
    ap.add_argument("--cols", type=int, default=1024)
    ap.add_argument("--outs", type=int, default=2816)
    ap.add_argument("--vocab", type=int, default=16384)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--dtype", choices=["f16", "bf16"], default="bf16")
    ap.add_argument("--lr", type=float, default=4.0)
    a = ap.parse_args(argv)
    dtype = torch.float16 if a.dtype == "f16" else torch.bfloat16
    gen = torch.Generator().manual_seed(1)
    x = torch.randn((a.rows, a.cols), generator=gen).to(dtype).cuda()
    targets = torch.randint(0, a.vocab, (a.rows,), generator=gen).cuda()
    block = GatedBlock(a.cols, a.outs, a.vocab, dtype)
    losses = []
    for i in range(a.steps):
        losses.append(float(step(block, x, targets, a.lr)))
        print(f"step {i:3d}  loss {losses[-1]:.5f}")
    return losses


if __name__ == "__main__":
    main()
