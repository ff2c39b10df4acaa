"""The operators between the norm and the loss in 64 bits on the CPU, and how far a result of the kernels may be
from them.

Bounds, element by element.  A product sums K exact products in fp32: with S the sum of their magnitudes it
is off by at most GAMMA(K) S, a unit of 2^-23 for each product (the tensor core truncates).  A rounding to a
type is off by half a step, finfo(t).eps / 2 of the value, or half the smallest subnormal.  Exponentials and
the division of the logistic function are good to 2^-19 of their value here (special-function unit; an
argument z, up to 32 in magnitude in the tests, is rounded by 2^-24 z first).
"""

import torch

F64 = torch.float64
FUNCTION = 2.0 ** -19


def gamma(k):
    return k * 2.0 ** -23


def rounding(ref, dtype):
    info = torch.finfo(dtype)
    return ref.abs() * (info.eps / 2) + info.smallest_normal * info.eps / 2


def kept(ref, dtype):
    """Rounding of what goes into a second product over the rows [rows, n]: up to 8 rows are kept in two
    terms, so that only the second one's rounding is left."""
    if ref.shape[0] > 8:
        return rounding(ref, dtype)
    info = torch.finfo(dtype)
    return ref.abs() * (info.eps / 2) ** 2 + info.smallest_normal * info.eps


def product(a, b):
    """(a b, sum of magnitudes)"""
    a, b = a.to(F64), b.to(F64)
    return a @ b, a.abs() @ b.abs()


def assert_within(got, ref, bound, what):
    got = got.detach().cpu().to(F64)
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= bound)
    if bad.any():
        at = bad.nonzero()[0].tolist()
        i = tuple(at)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {at}: "
                             f"{got[i].item()} against {ref[i].item()} +- {bound[i].item():.3g}")


def gate(g, act):
    """act(g) and act'(g).  GELU by the logistic function: 1 + tanh would leave nothing of s where g is
    below -6 (at -9 it is 1.5e-29)."""
    if act == "silu":
        s, slope = torch.sigmoid(g), 1.0
    else:
        c = 2 * (2 / torch.pi) ** 0.5
        s, slope = torch.sigmoid(c * (g + 0.044715 * g ** 3)), c * (1 + 3 * 0.044715 * g * g)
    return g * s, s + g * s * (1 - s) * slope


def gated(x, wg, wu, act):
    """{name: (value, bound)} of h, g and u."""
    k, dt = x.shape[1], x.dtype
    g, sg = product(x, wg)
    u, su = product(x, wu)
    a, _ = gate(g, act)
    dg, du = gamma(k) * sg, gamma(k) * su
    # |act'| <= 1.13; over a step dg act changes by at most that much of it
    dh = 1.13 * dg * (u.abs() + du) + (a.abs() + 1.13 * dg) * du + FUNCTION * (a * u).abs()
    return {"h": (a * u, rounding(a * u, dt) + dh * 1.01),
            "g": (g, rounding(g, dt) + dg * 1.01), "u": (u, rounding(u, dt) + du * 1.01)}


def gated_grads(dh, g, u, x, wg, wu, act):
    """{name: (value, bound)} of dx, dwg and dwu; dg and du are rounded on the way."""
    dt = dh.dtype
    dh, g, u, x, wg, wu = (t.to(F64) for t in (dh, g, u, x, wg, wu))
    a, slope = gate(g, act)
    dg, du = dh * u * slope, dh * a
    # act' is a sum of two terms of at most 1.2 (1 + |g|): its own error is relative to those
    eg = kept(dg, dt) + FUNCTION * (dh * u).abs() * 1.2 * (1 + g.abs())
    eu = kept(du, dt) + FUNCTION * du.abs()
    out = {}
    dx = dg @ wg.t() + du @ wu.t()
    s = dg.abs() @ wg.abs().t() + du.abs() @ wu.abs().t()
    e = eg @ wg.abs().t() + eu @ wu.abs().t()
    out["dx"] = (dx, rounding(dx, dt) + 1.02 * (e + gamma(2 * g.shape[1]) * s))
    for name, d, err in (("dwg", dg, eg), ("dwu", du, eu)):
        w = x.t() @ d
        out[name] = (w, rounding(w, dt) + 1.02 * (x.abs().t() @ err
                                                  + gamma(x.shape[0]) * (x.abs().t() @ d.abs())))
    return out


def xent(x, w, targets, ignore):
    """{name: (value, bound)} of loss and lse, [rows]."""
    logits, s = product(x, w.t())
    top = gamma(x.shape[1]) * s.max(dim=1).values      # no logit is further off
    lse = torch.logsumexp(logits, dim=1)
    valid = targets != ignore
    hit = logits.gather(1, targets.clamp(0, w.shape[0] - 1)[:, None])[:, 0]
    loss = torch.where(valid, lse - hit, 0.0)
    # sums of exponentials: 2^-19 each, and as much again for adding them up; then rounded twice
    e = top + 2 * FUNCTION + 2.0 ** -22 * lse.abs()
    return {"lse": (lse, e), "loss": (loss, torch.where(valid, e + top + 2.0 ** -22 * hit.abs(), 0.0))}


def xent_grads(dloss, x, w, targets, lse, ignore):
    """{name: (value, bound)} of dx and dw; the gradients of the logits are rounded on the way."""
    dt = x.dtype
    x, w, lse = x.to(F64), w.to(F64), lse.to(F64)
    logits, s = product(x, w.t())
    p = torch.exp(logits - lse[:, None])
    valid = targets != ignore
    weight = torch.where(valid, dloss.to(F64), 0.0)[:, None]
    hot = torch.zeros_like(p)
    hot.scatter_(1, targets.clamp(0, w.shape[0] - 1)[:, None], 1.0)
    d = (p - hot) * weight
    # a logit that is off by e makes p off by e p; weights are scaled and scaled back (2^-22); fp16
    # gradients are held relative to 2^15, so their smallest step is 2^-24-15 of the largest weight
    e = p * weight.abs() * (gamma(x.shape[1]) * s * 1.01 + FUNCTION) + d.abs() * 2.0 ** -22
    step = torch.finfo(dt).eps / 2
    e = e + d.abs() * (step if d.shape[0] > 8 else step ** 2) + weight.abs().max() * 2.0 ** -39
    out = {}
    dx = d @ w
    out["dx"] = (dx, rounding(dx, dt) + 1.02 * (e @ w.abs() + gamma(w.shape[0]) * (d.abs() @ w.abs())))
    dw = d.t() @ x
    out["dw"] = (dw, rounding(dw, dt) + 1.02 * (e.t() @ x.abs()
                                                + gamma(x.shape[0]) * (d.abs().t() @ x.abs())))
    return out
