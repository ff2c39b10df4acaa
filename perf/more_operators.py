"""The operators between the norm and the loss of a language model's training step, case by case: the
gated feed-forward projections and their gradients, the cross entropy of a vocabulary projection and
its gradients, and a linear layer's input gradient.

``run`` computes each operator in elementary torch operations in 32 bits (``own`` false) or by the
library's entry points (``own`` true); ``exact`` computes it from its definition in 64 bits.

    gated_fwd    h = act(g) u,  g = x Wg,  u = x Wu          x [rows, cols], Wg, Wu [cols, outs]
    gated_bwd    dx, dWg, dWu from dh, with g and u as the forward pass kept them
    xent_fwd     loss = lse - logit[target], lse = log sum exp logits,  logits = x W^T, W [vocab, cols]
    xent_bwd     dx, dW from the gradient of each row's loss, with lse as the forward pass gave it
    input_grad   dx = dy W^T                                 dy [rows, outs], W [cols, outs]

act is SiLU, g s(g), or GELU in its tanh form, g s(2 sqrt(2 / pi) (g + 0.044715 g^3)), s the logistic
function.  Rows whose target is IGNORE have no loss and no gradient.
"""

import math

import torch

own = False

IGNORE = -100
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
SIZE = 2
GELU_A, GELU_B = 2.0 * math.sqrt(2.0 / math.pi), 0.044715


def listed():
    return [
        # one token of a reply through a small and through a large layer: latency, then the weights' bytes
        {"name": "gated_fwd_1x1024x2048_f16", "op": "gated_fwd", "rows": 1, "cols": 1024, "outs": 2048, "dtype": "f16", "act": "silu", "keep": False},
        {"name": "gated_fwd_4x4096x8192_bf16", "op": "gated_fwd", "rows": 4, "cols": 4096, "outs": 8192, "dtype": "bf16", "act": "silu", "keep": False},
        # a ragged batch without gradients
        {"name": "gated_fwd_1001x1000x2728_f16", "op": "gated_fwd", "rows": 1001, "cols": 1000, "outs": 2728, "dtype": "f16", "act": "gelu", "keep": False},
        # a training step's forward pass: g and u are kept for the backward pass
        {"name": "gated_fwd_keep_8192x4096x8192_bf16", "op": "gated_fwd", "rows": 8192, "cols": 4096, "outs": 8192, "dtype": "bf16", "act": "silu", "keep": True},
        # the same step's backward pass, and a small ragged one
        {"name": "gated_bwd_8192x4096x8192_bf16", "op": "gated_bwd", "rows": 8192, "cols": 4096, "outs": 8192, "dtype": "bf16", "act": "silu"},
        {"name": "gated_bwd_333x1000x2008_f16", "op": "gated_bwd", "rows": 333, "cols": 1000, "outs": 2008, "dtype": "f16", "act": "gelu"},
        # the loss of a short text under a small model, and of a training step with a large vocabulary
        {"name": "xent_fwd_61x1024x32001_f16", "op": "xent_fwd", "rows": 61, "cols": 1024, "vocab": 32001, "dtype": "f16"},
        {"name": "xent_fwd_4096x4096x65536_bf16", "op": "xent_fwd", "rows": 4096, "cols": 4096, "vocab": 65536, "dtype": "bf16"},
        # and their gradients
        {"name": "xent_bwd_250x1024x10007_f16", "op": "xent_bwd", "rows": 250, "cols": 1024, "vocab": 10007, "dtype": "f16"},
        {"name": "xent_bwd_4096x4096x65536_bf16", "op": "xent_bwd", "rows": 4096, "cols": 4096, "vocab": 65536, "dtype": "bf16"},
        # what a linear layer hands back: few tokens, and the largest square problem
        {"name": "input_grad_16x2048x8192_bf16", "op": "input_grad", "rows": 16, "cols": 2048, "outs": 8192, "dtype": "bf16"},
        {"name": "input_grad_8192x8192x8192_bf16", "op": "input_grad", "rows": 8192, "cols": 8192, "outs": 8192, "dtype": "bf16"},
    ]


# how far each operator's listed cases go, in multiplications of one of its products
LARGEST = {"gated_fwd": 1 << 38, "gated_bwd": 1 << 38, "xent_fwd": 1 << 40, "xent_bwd": 1 << 40, "input_grad": 1 << 39}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["gated_fwd", "gated_bwd", "xent_fwd", "xent_bwd", "input_grad"])
    while True:
        case = {"op": op, "rows": _log_int(rng, 1, 8192), "cols": 8 * _log_int(rng, 16, 1024), "dtype": rng.choice(["f16", "bf16"])}
        if op.startswith("xent"):
            case["vocab"] = _log_int(rng, 500, 65536)
            over = case["vocab"]
        else:
            case["outs"] = 8 * _log_int(rng, 16, 1024)
            over = case["outs"]
        if op.startswith("gated"):
            case["act"] = rng.choice(["silu", "gelu"])
        if op == "gated_fwd":
            case["keep"] = rng.random() < 0.5
        if case["rows"] * case["cols"] * over <= LARGEST[op]:
            return case


def _normal(shape, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, rows, cols, dt = case["op"], case["rows"], case["cols"], DTYPES[case["dtype"]]
    state = {"case": case, "dtype": dt}
    if op == "input_grad":
        state["dy"] = _normal((rows, case["outs"]), gen, 0.05).to(dt)
        state["w"] = _normal((cols, case["outs"]), gen, case["outs"] ** -0.5).to(dt)
        return state
    # a norm's output: unit variance, channels of unequal size
    x = _normal((rows, cols), gen).mul_(torch.exp(0.3 * _normal((cols,), gen)))
    if op.startswith("gated"):
        outs = case["outs"]
        state["x"] = x.to(dt)
        state["wg"] = _normal((cols, outs), gen, 1.5 * cols ** -0.5).to(dt)
        state["wu"] = _normal((cols, outs), gen, cols ** -0.5).to(dt)
        if op == "gated_bwd":
            state["g"] = (state["x"].float() @ state["wg"].float()).to(dt)
            state["u"] = (state["x"].float() @ state["wu"].float()).to(dt)
            state["dh"] = _normal((rows, outs), gen, 0.05).to(dt)
        return state
    vocab = case["vocab"]
    w = _normal((vocab, cols), gen, 2.0 * cols ** -0.5)
    # frequent words first; a model that is part of the way: x leans towards its target's row
    targets = (vocab ** torch.rand(rows, generator=gen, device="cuda")).long().sub_(1).clamp_(0, vocab - 1)
    lean = 3.0 * torch.rand((rows, 1), generator=gen, device="cuda")
    state["x"] = x.add_(w[targets] * lean).to(dt)
    state["w"] = w.to(dt)
    state["targets"] = torch.where(torch.rand(rows, generator=gen, device="cuda") < 0.06, IGNORE, targets)   # padding
    if op == "xent_bwd":
        logits = state["x"].float() @ state["w"].float().t()
        top = logits.amax(dim=1)
        state["lse"] = top + torch.log(logits.sub_(top[:, None]).exp_().sum(dim=1))
        valid = state["targets"] != IGNORE
        state["dloss"] = valid.float() / valid.sum().clamp_min(1)   # of the mean
    return state


def _gate(g, act):
    """act(g) and its derivative in 32 bits."""
    z = g if act == "silu" else GELU_A * (g + GELU_B * (g * g * g))
    s = 1.0 / (1.0 + torch.exp(-z))
    slope = 1.0 if act == "silu" else GELU_A * (1.0 + 3.0 * GELU_B * (g * g))
    return g * s, s + g * s * (1.0 - s) * slope


def _plain(st):
    case, dt = st["case"], st["dtype"]
    op = case["op"]
    if op == "input_grad":
        return (st["dy"].float() @ st["w"].float().t()).to(dt)
    x = st["x"].float()
    if op == "gated_fwd":
        g, u = x @ st["wg"].float(), x @ st["wu"].float()
        out = {"h": (_gate(g, case["act"])[0] * u).to(dt)}
        if case["keep"]:
            out["g"], out["u"] = g.to(dt), u.to(dt)
        return out
    if op == "gated_bwd":
        dh = st["dh"].float()
        a, slope = _gate(st["g"].float(), case["act"])
        dg, du = dh * st["u"].float() * slope, dh * a
        dx = dg @ st["wg"].float().t() + du @ st["wu"].float().t()
        return {"dx": dx.to(dt), "dwg": (x.t() @ dg).to(dt), "dwu": (x.t() @ du).to(dt)}
    w, targets = st["w"].float(), st["targets"]
    valid = targets != IGNORE
    at = torch.where(valid, targets, 0)[:, None]
    logits = x @ w.t()
    if op == "xent_fwd":
        top = logits.amax(dim=1)
        hit = logits.gather(1, at)[:, 0]
        lse = top + torch.log(torch.exp(logits - top[:, None]).sum(dim=1))
        return {"loss": torch.where(valid, lse - hit, 0.0), "lse": lse}
    dlogits = torch.exp(logits - st["lse"][:, None])
    dlogits.scatter_add_(1, at, -torch.ones_like(st["lse"])[:, None])
    dlogits *= torch.where(valid, st["dloss"], 0.0)[:, None]
    return {"dx": (dlogits @ w).to(dt), "dw": (dlogits.t() @ x).to(dt)}


def run(state):
    if not own:
        return _plain(state)
    import persistent_warp_specialized_gb300 as tg

    case = state["case"]
    op = case["op"]
    if op == "input_grad":
        return tg.input_grad(state["dy"], state["w"])
    if op == "gated_fwd":
        if not case["keep"]:
            return {"h": tg.gated_forward(state["x"], state["wg"], state["wu"], act=case["act"])}
        h, g, u = tg.gated_forward(state["x"], state["wg"], state["wu"], act=case["act"], keep=True)
        return {"h": h, "g": g, "u": u}
    if op == "gated_bwd":
        dx, dwg, dwu = tg.gated_backward(state["dh"], state["g"], state["u"], state["x"], state["wg"], state["wu"], act=case["act"])
        return {"dx": dx, "dwg": dwg, "dwu": dwu}
    if op == "xent_fwd":
        loss, lse = tg.linear_cross_entropy(state["x"], state["w"], state["targets"], ignore_index=IGNORE)
        return {"loss": loss, "lse": lse}
    dx, dw = tg.linear_cross_entropy_backward(state["dloss"], state["x"], state["w"], state["targets"], state["lse"], ignore_index=IGNORE)
    return {"dx": dx, "dw": dw}


def work(case):
    rows, cols, op = case["rows"], case["cols"], case["op"]
    if op.startswith("xent"):
        n, io = rows * cols * case["vocab"], SIZE * cols * (rows + case["vocab"])
        if op == "xent_fwd":
            return {"bytes": io + 16 * rows, "flops": 2 * n}
        return {"bytes": 2 * io + 16 * rows, "flops": 6 * n}    # the logits again, dx and dw
    n, weights, x, h = rows * cols * case["outs"], SIZE * cols * case["outs"], SIZE * rows * cols, SIZE * rows * case["outs"]
    if op == "input_grad":
        return {"bytes": weights + x + h, "flops": 2 * n}
    if op == "gated_fwd":
        return {"bytes": 2 * weights + x + (3 if case["keep"] else 1) * h, "flops": 4 * n}
    return {"bytes": 4 * weights + 2 * x + 3 * h, "flops": 8 * n}


def _gate64(g, act):
    """act and its derivative by the logistic function of torch in 64 bits."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + GELU_B * g ** 3))
    return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t * t) * c * (1 + 3 * GELU_B * g * g) / 2


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "input_grad":
        return torch.einsum("to,co->tc", st["dy"].double(), st["w"].double())
    x = st["x"].double()
    if op == "gated_fwd":
        g, u = x.matmul(st["wg"].double()), x.matmul(st["wu"].double())
        out = {"h": _gate64(g, case["act"])[0].mul_(u)}
        if case["keep"]:
            out.update(g=g, u=u)
        return out
    if op == "gated_bwd":
        a, slope = _gate64(st["g"].double(), case["act"])
        dh = st["dh"].double()
        du, dg = dh * a, slope.mul_(dh).mul_(st["u"].double())
        dx = torch.einsum("to,co->tc", dg, st["wg"].double()).add_(torch.einsum("to,co->tc", du, st["wu"].double()))
        return {"dx": dx, "dwg": torch.einsum("tc,to->co", x, dg), "dwu": torch.einsum("tc,to->co", x, du)}
    w, targets = st["w"].double(), st["targets"]
    logits = torch.einsum("tc,vc->tv", x, w)
    kept = targets.ge(0)
    if op == "xent_fwd":
        lse = torch.logsumexp(logits, dim=1)
        rows = torch.arange(len(targets), device=targets.device)
        return {"loss": (lse - logits[rows, targets.clamp(min=0)]) * kept, "lse": lse}
    p = logits.sub_(st["lse"].double()[:, None]).exp_()
    rows = kept.nonzero()[:, 0]
    p[rows, targets[rows]] -= 1
    p.mul_((st["dloss"].double() * kept)[:, None])
    return {"dx": torch.einsum("tv,vc->tc", p, w), "dw": torch.einsum("tv,tc->vc", p, x)}
