"""The training operators around the GEMM, case by case: layer norm forward and backward, activation
checkpoints in 8 bits, and the weight gradient taken from a checkpoint.

``run`` computes each operator in elementary torch operations in 32 bits (``own`` false) or by the
library's entry points (``own`` true); ``exact`` computes it from its definition in 64 bits.

A checkpoint of x [rows, cols] holds E4M3 bytes q [rows, 32 ceil(cols / 32)] (zeros past ``cols``) and
one E8M0 byte per 32 values, s [rows, ceil(cols / 32)]; it stands for q * 2^(s - 127).  The scale of a
block is 2^(floor(log2 amax) - 8), with the exponent clamped to [-127, 127].
"""

import torch

own = False

EPS = 1e-5
BLOCK = 32
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"f16": 2, "bf16": 2, "f32": 4}
# what a norm's kept output is read back as: both hold every value of a checkpoint of that type
KEPT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.bfloat16}


def listed():
    return [
        # a few tokens being generated: latency
        {"name": "ln_fwd_4x1024_f16", "op": "ln_fwd", "rows": 4, "cols": 1024, "dtype": "f16", "ckpt": False},
        # a training step's norm at the width of the 4096 problems
        {"name": "ln_fwd_8192x4096_bf16", "op": "ln_fwd", "rows": 8192, "cols": 4096, "dtype": "bf16", "ckpt": False},
        # the ragged problem's sizes, with the output kept in 8 bits for the backward pass
        {"name": "ln_fwd_ckpt_4000x7000_bf16", "op": "ln_fwd", "rows": 4000, "cols": 7000, "dtype": "bf16", "ckpt": True},
        # the largest norm: the width of the 8192 problems
        {"name": "ln_bwd_8192x8192_bf16", "op": "ln_bwd", "rows": 8192, "cols": 8192, "dtype": "bf16", "ckpt": False},
        # the norm's input was kept in 8 bits
        {"name": "ln_bwd_ckpt_8192x4096_f16", "op": "ln_bwd", "rows": 8192, "cols": 4096, "dtype": "f16", "ckpt": True},
        # a residual stream in 32 bits, odd sizes: rows that no vector load is aligned to
        {"name": "ln_bwd_1001x2047_f32", "op": "ln_bwd", "rows": 1001, "cols": 2047, "dtype": "f32", "ckpt": False},
        # small and large checkpoints, there and back
        {"name": "ckpt_256x256_f16", "op": "ckpt", "rows": 256, "cols": 256, "dtype": "f16"},
        {"name": "ckpt_8192x8192_bf16", "op": "ckpt", "rows": 8192, "cols": 8192, "dtype": "bf16"},
        # weight gradients: the smallest square problem, the ragged one, the largest, and one with
        # few output tiles and many tokens
        {"name": "wgrad_256x256x256_f16", "op": "wgrad", "rows": 256, "cols": 256, "outs": 256, "dtype": "f16"},
        {"name": "wgrad_4000x2048x7000_bf16", "op": "wgrad", "rows": 4000, "cols": 2048, "outs": 7000, "dtype": "bf16"},
        {"name": "wgrad_8192x8192x8192_bf16", "op": "wgrad", "rows": 8192, "cols": 8192, "outs": 8192, "dtype": "bf16"},
        {"name": "wgrad_32768x1000x512_bf16", "op": "wgrad", "rows": 32768, "cols": 1000, "outs": 512, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "ckpt", "wgrad"])
    if op == "wgrad":
        while True:
            case = {"op": op, "rows": _log_int(rng, 1, 32768), "cols": _log_int(rng, 16, 8192),
                    "outs": 8 * _log_int(rng, 1, 1024), "dtype": rng.choice(["f16", "bf16"])}
            if case["rows"] * case["cols"] * case["outs"] <= 1 << 38:
                return case
    while True:
        case = {"op": op, "rows": _log_int(rng, 1, 32768), "cols": _log_int(rng, 16, 16384),
                "dtype": rng.choice(["f16", "bf16", "f32"])}
        if op != "ckpt":
            case["ckpt"] = rng.random() < 0.4
        if case["rows"] * case["cols"] <= 1 << 26:
            return case


def _blocks(cols):
    return (cols + BLOCK - 1) // BLOCK


def _activations(rows, cols, gen):
    """Activations as a norm meets them: channels of unequal size, a few of them large, off zero."""
    scale = torch.exp(0.5 * torch.randn(cols, generator=gen, device="cuda"))
    shift = 0.3 + 0.2 * torch.randn(cols, generator=gen, device="cuda")
    large = torch.rand(cols, generator=gen, device="cuda") < 0.003
    scale = torch.where(large, 10.0 * scale, scale)
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    return x.mul_(scale).add_(shift)


def _pack(x):
    """The checkpoint of x: blocks of 32 in 32 bits."""
    rows, cols = x.shape
    nb = _blocks(cols)
    b = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    amax = b.abs().amax(dim=2)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 9, -127).clamp_(-127, 127)
    q = (b * torch.exp2(-e.float())[:, :, None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(rows, nb * BLOCK), (e + 127).to(torch.uint8)


def _unpack(q, s, cols):
    """The values a checkpoint stands for, in 32 bits (exact)."""
    rows, nb = s.shape
    v = q.view(torch.float8_e4m3fn).float().view(rows, nb, BLOCK)
    return (v * torch.exp2(s.float() - 127.0)[:, :, None]).view(rows, nb * BLOCK)[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
    state = {"case": case, "dtype": dt, "cols": cols}
    x = _activations(rows, cols, gen)
    if case["op"] == "wgrad":
        # what a norm's output looks like: unit variance in each row
        x = (x - x.mean(dim=1, keepdim=True)) / x.std(dim=1, keepdim=True, unbiased=False).add_(EPS)
        state["q"], state["s"] = _pack(x.to(dt))
        state["dy"] = torch.randn((rows, case["outs"]), generator=gen, device="cuda").mul_(0.05).to(dt)
        return state
    state["x"] = x.to(dt)
    if case["op"] == "ckpt":
        return state
    state["gamma"] = 1.0 + 0.1 * torch.randn(cols, generator=gen, device="cuda")
    state["beta"] = 0.1 * torch.randn(cols, generator=gen, device="cuda")
    if case["op"] == "ln_bwd":
        state["dy"] = torch.randn((rows, cols), generator=gen, device="cuda").mul_(0.05).to(dt)
        xf = state["x"].double()
        mean = xf.mean(dim=1)
        state["mean"] = mean.float()
        state["rstd"] = torch.rsqrt((xf - mean[:, None]).square().mean(dim=1) + EPS).float()
        if case["ckpt"]:
            state["q"], state["s"] = _pack(state.pop("x"))
    return state


def _plain(st):
    op, dt, cols = st["case"]["op"], st["dtype"], st["cols"]
    if op == "wgrad":
        return (_unpack(st["q"], st["s"], cols).t() @ st["dy"].float()).to(dt)
    if op == "ckpt":
        q, s = _pack(st["x"])
        return _unpack(q, s, cols).to(dt)
    if op == "ln_fwd":
        x = st["x"].float()
        mean = x.mean(dim=1)
        c = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((c * c).mean(dim=1) + EPS)
        y = (c * rstd[:, None] * st["gamma"] + st["beta"]).to(dt)
        out = {"y": y, "mean": mean, "rstd": rstd}
        if st["case"]["ckpt"]:
            q, s = _pack(y)
            out["kept"] = _unpack(q, s, cols).to(KEPT[st["case"]["dtype"]])
        return out
    x = _unpack(st["q"], st["s"], cols) if st["case"]["ckpt"] else st["x"].float()
    dy = st["dy"].float()
    xh = (x - st["mean"][:, None]) * st["rstd"][:, None]
    g = dy * st["gamma"]
    dx = st["rstd"][:, None] * (g - g.mean(dim=1, keepdim=True) - xh * (g * xh).mean(dim=1, keepdim=True))
    return {"dx": dx.to(dt), "dgamma": (dy * xh).sum(dim=0), "dbeta": dy.sum(dim=0)}


def run(state):
    if not own:
        return _plain(state)
    import persistent_warp_specialized_gb300 as tg

    op = state["case"]["op"]
    if op == "wgrad":
        return tg.ckpt8_wgrad(tg.Checkpoint8(state["q"], state["s"], state["cols"]), state["dy"])
    if op == "ckpt":
        return tg.ckpt8_unpack(tg.ckpt8_pack(state["x"]), state["dtype"])
    if op == "ln_fwd":
        if not state["case"]["ckpt"]:
            y, mean, rstd = tg.layer_norm(state["x"], state["gamma"], state["beta"], EPS)
            return {"y": y, "mean": mean, "rstd": rstd}
        y, mean, rstd, kept = tg.layer_norm(state["x"], state["gamma"], state["beta"], EPS, checkpoint=True)
        return {"y": y, "mean": mean, "rstd": rstd, "kept": tg.ckpt8_unpack(kept, KEPT[state["case"]["dtype"]])}
    x = tg.Checkpoint8(state["q"], state["s"], state["cols"]) if state["case"]["ckpt"] else state["x"]
    dx, dgamma, dbeta = tg.layer_norm_backward(state["dy"], x, state["mean"], state["rstd"], state["gamma"])
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def work(case):
    rows, cols, e, op = case["rows"], case["cols"], SIZES[case["dtype"]], case["op"]
    n = rows * cols
    kept = rows * _blocks(cols) * (BLOCK + 1)       # bytes of a checkpoint
    if op == "wgrad":
        return {"bytes": kept + e * (rows + cols) * case["outs"], "flops": 2 * n * case["outs"]}
    if op == "ckpt":                                # x in; the checkpoint out and in again; values out
        return {"bytes": 2 * e * n + 2 * kept, "flops": 4 * n}
    if op == "ln_fwd":
        extra = 2 * kept + 2 * n if case["ckpt"] else 0
        return {"bytes": 2 * e * n + 8 * cols + 8 * rows + extra, "flops": 8 * n}
    return {"bytes": (kept if case["ckpt"] else e * n) + 2 * e * n + 12 * cols + 8 * rows, "flops": 14 * n}


def _kept64(v):
    """The values a checkpoint of v (64 bits) stands for: per block of 32, the E4M3 grid scaled by 2^e."""
    rows, cols = v.shape
    out = torch.empty_like(v)
    for c0 in range(0, cols, BLOCK * 64):           # a slab of columns at a time, to bound memory
        slab = v[:, c0:c0 + BLOCK * 64]
        w = slab.shape[1]
        full = torch.zeros((rows, _blocks(w) * BLOCK), dtype=v.dtype, device=v.device)
        full[:, :w] = slab
        block = full.view(rows, -1, BLOCK)
        top = block.abs().max(dim=2, keepdim=True).values
        e = torch.frexp(torch.where(top > 0, top, 2.0 ** -200)).exponent - 1 - 8
        unit = torch.exp2(e.clamp(-127, 127).double())
        u = block / unit
        step = torch.exp2(torch.frexp(u.abs().clamp_min(2.0 ** -6)).exponent.double() - 1 - 3)
        u = torch.minimum(torch.round(u / step) * step, torch.tensor(448.0, dtype=v.dtype, device=v.device))
        u = u.clamp_min(-448.0)
        out[:, c0:c0 + w] = (u * unit).view(rows, -1)[:, :w]
    return out


def _stands_for64(q, s, cols):
    """E4M3 and E8M0 bytes as 64-bit values, from the bit fields."""
    b = q.to(torch.int64)
    sign = 1.0 - 2.0 * (b >> 7).double()
    exp, frac = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(exp > 0, (8 + frac) * torch.exp2(exp.double() - 10), frac * 2.0 ** -9)
    unit = torch.exp2(s.double() - 127).repeat_interleave(BLOCK, dim=1)
    return (sign * mag * unit)[:, :cols]


def exact(case, seed):
    st = prepare(case, seed)
    op, cols = case["op"], case["cols"]
    if op == "wgrad":
        return _stands_for64(st["q"], st["s"], cols).T.matmul(st["dy"].double())
    if op == "ckpt":
        return _kept64(st["x"].double())
    gamma, beta = st["gamma"].double(), st["beta"].double()
    if op == "ln_fwd":
        x = st["x"].double()
        var, mean = torch.var_mean(x, dim=1, unbiased=False)
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(beta, (x - mean[:, None]).mul_(rstd[:, None]), gamma)
        out = {"y": y, "mean": mean, "rstd": rstd}
        if case["ckpt"]:                            # what is kept is the output as it was rounded
            out["kept"] = _kept64(y.to(st["dtype"]).double())
        return out
    x = _stands_for64(st["q"], st["s"], cols) if case["ckpt"] else st["x"].double()
    mean, rstd = st["mean"].double()[:, None], st["rstd"].double()[:, None]
    dy = st["dy"].double()
    xh = (x - mean) * rstd
    dgamma, dbeta = torch.einsum("tc,tc->c", dy, xh), dy.sum(dim=0)
    g = dy * gamma
    a, b = g.sum(dim=1, keepdim=True) / cols, torch.einsum("tc,tc->t", g, xh)[:, None] / cols
    return {"dx": rstd * (g - a - xh * b), "dgamma": dgamma, "dbeta": dbeta}
