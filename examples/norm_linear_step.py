"""Trains one pre-norm linear layer, z = layer_norm(x) W, keeping its activations in 8 bits.

    python examples/norm_linear_step.py [--rows 4096 --cols 2048 --outs 2048 --steps 20 --dtype bf16]

The forward pass packs x and y = layer_norm(x) to 8 bits as it goes and drops both; the backward pass
takes the weight gradient from y's checkpoint and the norm's gradients from x's.  The product with W is
the dense GEMM's; the gradient towards y reads W as it lies (input_grad).  Needs a GB300 and the built
library (see the README).
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import persistent_warp_specialized_gb300 as tg


class NormLinear:
    """gamma, beta [cols] and W [cols, outs]; master copies in float32."""

    def __init__(self, cols, outs, dtype, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.dtype = dtype
        self.gamma = torch.ones(cols, device="cuda")
        self.beta = torch.zeros(cols, device="cuda")
        self.w = (torch.randn((cols, outs), generator=gen) / cols ** 0.5).cuda()

    def forward(self, x):
        """z, and what the backward pass needs: checkpoints of x and y, and the row statistics."""
        y, mean, rstd, kept_y = tg.layer_norm(x, self.gamma, self.beta, checkpoint=True)
        z = tg.gemm(y, self.w.to(self.dtype))
        return z, (tg.ckpt8_pack(x), kept_y, mean, rstd)

    def backward(self, dz, saved):
        """(dx, dgamma, dbeta, dw) from dz [rows, outs]."""
        kept_x, kept_y, mean, rstd = saved
        dw = tg.ckpt8_wgrad(kept_y, dz)
        dy = tg.input_grad(dz, self.w.to(self.dtype))
        dx, dgamma, dbeta = tg.layer_norm_backward(dy, kept_x, mean, rstd, self.gamma)
        return dx, dgamma, dbeta, dw


def step(layer, x, target, lr):
    """One step of gradient descent on the mean square of z - target; returns the loss."""
    z, saved = layer.forward(x)
    diff = z.float() - target
    loss = diff.square().mean()
    # of the sum, to keep 16-bit gradients in range; a weight meets rows results, gamma and beta all
    dx, dgamma, dbeta, dw = layer.backward((2 * diff).to(layer.dtype), saved)
    layer.w -= lr / diff.shape[0] * dw.float()
    layer.gamma -= lr / diff.numel() * dgamma
    layer.beta -= lr / diff.numel() * dbeta
    return loss


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=4096)
    ap.add_argument("--cols", type=int, default=2048)
    ap.add_argument("--outs", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--dtype", choices=["f16", "bf16"], default="bf16")
    ap.add_argument("--lr", type=float, default=0.15)
    a = ap.parse_args(argv)
    dtype = torch.float16 if a.dtype == "f16" else torch.bfloat16
    gen = torch.Generator().manual_seed(1)
    x = (torch.randn((a.rows, a.cols), generator=gen) + 0.5).to(dtype).cuda()
    layer = NormLinear(a.cols, a.outs, dtype)
    teacher = NormLinear(a.cols, a.outs, dtype, seed=7)
    target = teacher.forward(x)[0].float()
    losses = []
    for i in range(a.steps):
        losses.append(float(step(layer, x, target, a.lr)))
        print(f"step {i:3d}  loss {losses[-1]:.5f}")
    kept = sum(k.q.numel() + k.s.numel() for k in layer.forward(x)[1][:2])
    print(f"activations kept: {kept / 2 ** 20:.1f} MiB in 8 bits, "
          f"{2 * x.numel() * x.element_size() / 2 ** 20:.1f} MiB in 16")
    return losses


if __name__ == "__main__":
    main()
