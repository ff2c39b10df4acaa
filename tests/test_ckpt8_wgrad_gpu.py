"""The weight gradient from an 8-bit checkpoint against the binary64 oracle.

Integer cases are bit-exact: every product and partial sum is an integer below 2^24.  Elsewhere the
bound is fixed before the first run: the kernel sums T exact products in fp32, where the tensor core
may truncate (2^-23 of the running magnitude for each add), joins the ranges in fp32, and rounds once:
    |dW - ref| <= T 2^-23 (|x|^T |dY|) + half an ulp of the result.
"""

import numpy as np
import pytest
import torch

import persistent_warp_specialized_gb300 as tg
from gpu_helpers import ensure_library
from oracle import train

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}
INT_BYTES = torch.tensor([0xC8, 0xC4, 0xC0, 0xB8, 0x00, 0x38, 0x40, 0x44, 0x48], dtype=torch.uint8)


@pytest.fixture(scope="module", autouse=True)
def library():
    ensure_library()


def f64(t):
    return t.detach().cpu().double().numpy()


def integers(rows, cols, outs, dtype, seed):
    """Checkpoint elements -4 .. 4 with scales 1 or 2, gradients -2 .. 2."""
    gen = torch.Generator().manual_seed(seed)
    nb = -(-cols // 32)
    q = INT_BYTES[torch.randint(0, 9, (rows, 32 * nb), generator=gen)]
    q[:, cols:] = 0
    s = torch.randint(127, 129, (rows, nb), generator=gen).to(torch.uint8)
    dy = torch.randint(-2, 3, (rows, outs), generator=gen).to(DT[dtype])
    return q, s, dy


def reference(q, s, cols, dy):
    return train.weight_gradient(q.numpy(), s.numpy(), cols, f64(dy))


def run(q, s, cols, dy, **kw):
    out = torch.full((cols, dy.shape[1]), float("nan"), dtype=dy.dtype, device="cuda")
    got = tg.ckpt8_wgrad(tg.Checkpoint8(q.cuda(), s.cuda(), cols), dy.cuda(), out=out, **kw)
    torch.cuda.synchronize()
    assert tg.tg_device_status() == 0
    return got


SHAPES = [(1, 1, 8), (1, 300, 264), (7, 33, 8), (63, 128, 128), (64, 129, 256), (65, 31, 512),
          (100, 256, 136), (256, 256, 256), (300, 1000, 72), (513, 257, 520), (1000, 64, 1024),
          (5000, 130, 200), (20000, 40, 16), (2048, 700, 2056), (700, 2500, 2304), (130, 5000, 4096)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols,outs", SHAPES)
def test_integers_bit_exact(rows, cols, outs, dtype):
    q, s, dy = integers(rows, cols, outs, dtype, rows + cols + outs)
    want = torch.from_numpy(reference(q, s, cols, dy)).to(DT[dtype])
    assert torch.equal(run(q, s, cols, dy).cpu(), want)


def check_close(got, q, s, cols, dy, dtype):
    x = train.unpack(q.numpy(), s.numpy(), cols)
    ref = x.T @ f64(dy)
    tol = x.shape[0] * 2.0 ** -23 * (np.abs(x).T @ np.abs(f64(dy)))
    err = np.abs(f64(got) - ref)
    bad = err > tol + (np.abs(ref) + tol) * HALF_ULP[dtype] + TINY[dtype]
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), err.max())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols,outs", [(3, 65, 24), (500, 300, 264), (4000, 513, 128),
                                            (30000, 100, 64), (1024, 1536, 1024)])
def test_packed_activations(rows, cols, outs, dtype):
    gen = torch.Generator().manual_seed(rows)
    x = torch.randn((rows, cols), generator=gen) * torch.exp(torch.randn(cols, generator=gen))
    kept = tg.ckpt8_pack(x.to(DT[dtype]).cuda())
    dy = (0.1 * torch.randn((rows, outs), generator=gen)).to(DT[dtype])
    q, s = kept.q.cpu(), kept.s.cpu()
    got = tg.ckpt8_wgrad(kept, dy.cuda())
    check_close(got, q, s, cols, dy, dtype)
    for _ in range(2):                           # sums are added in a fixed order
        assert torch.equal(tg.ckpt8_wgrad(kept, dy.cuda()), got)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_every_byte_under_every_scale(dtype):
    # dY = identity: dW is x itself, rounded once to the type.  Elements that are NaN, and scales
    # under which an element leaves the type's range (inf * 0 is NaN), are left out.
    fine = torch.tensor([i for i in range(256) if i & 0x7F != 0x7F]).to(torch.uint8)    # 254
    scales = torch.arange(255, dtype=torch.int32).to(torch.uint8)
    q = torch.cat([fine, torch.zeros(2, dtype=torch.uint8)]).repeat(255, 1)
    s = scales[:, None].repeat(1, 8).contiguous()
    x = torch.from_numpy(train.unpack(q.numpy(), s.numpy(), 254)).to(DT[dtype])
    keep = torch.isfinite(x).all(dim=1)
    q, s, x = q[keep], s[keep], x[keep]
    n = x.shape[0]
    assert n > 130
    got = run(q, s, 254, torch.eye(n, 256, dtype=DT[dtype]))
    assert torch.equal(got[:, :n].cpu(), x.t()) and (got[:, n:] == 0).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_what_is_not_finite_reaches_its_own_results(dtype):
    q, s, dy = integers(200, 96, 64, dtype, 5)
    q[17, 40] = 0x7F                             # an element's NaN: column 40 of x
    s[33, 0] = 255                               # a scale's NaN: columns 0..31
    dy[50, 9] = float("inf")                     # an infinite gradient: column 9 of dW
    got = run(q, s, 96, dy).cpu()
    nan = torch.isnan(got)
    bad_rows = set(range(32)) | {40}
    assert nan[sorted(bad_rows)].all()
    rest = [i for i in range(96) if i not in bad_rows]
    assert not nan[rest][:, [j for j in range(64) if j != 9]].any()
    assert (~torch.isfinite(got[rest][:, 9])).all()
    q[17, 40], s[33, 0] = 0x38, 127
    dy[50, 9] = 1.0
    want = torch.from_numpy(reference(q, s, 96, dy)).to(DT[dtype])
    cols = [j for j in range(64) if j != 9]
    keep = [i for i in rest]
    assert torch.equal(got[keep][:, cols], want[keep][:, cols])


def test_large_scales_take_the_long_way():
    # bf16, scales to 2^100 and elements up to 448 (past what one multiplication reaches)
    gen = torch.Generator().manual_seed(3)
    q = torch.randint(0, 0x7F, (128, 64), generator=gen).to(torch.uint8)
    s = torch.randint(100, 228, (128, 2), generator=gen).to(torch.uint8)
    dy = torch.zeros((128, 64), dtype=torch.bfloat16)
    dy[torch.arange(64), torch.arange(64)] = 1.0       # dW[:, t] is x[t]
    want = torch.from_numpy(train.unpack(q.numpy(), s.numpy(), 64)[:64]).to(torch.bfloat16).t()
    assert torch.equal(run(q, s, 64, dy).cpu(), want)


@pytest.mark.parametrize("pad_y,pad_w", [(8, 0), (0, 24), (64, 8)])
def test_row_strides(pad_y, pad_w):
    rows, cols, outs = 333, 190, 200
    q, s, dy = integers(rows, cols, outs, "bf16", 7)
    big = torch.full((rows, outs + pad_y), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = big[:, :outs]
    view.copy_(dy)
    whole = torch.full((cols, outs + pad_w), float("nan"), dtype=torch.bfloat16, device="cuda")
    kept = tg.Checkpoint8(q.cuda(), s.cuda(), cols)
    tg.ckpt8_wgrad(kept, view, out=whole[:, :outs])
    assert torch.equal(whole[:, :outs].cpu(), torch.from_numpy(reference(q, s, cols, dy)).bfloat16())
    assert torch.isnan(whole[:, outs:]).all()
    # and with the rows split (long contraction, one tile)
    q, s, dy = integers(9000, 60, 64, "bf16", 8)
    whole = torch.full((60, 64 + pad_w), float("nan"), dtype=torch.bfloat16, device="cuda")
    tg.ckpt8_wgrad(tg.Checkpoint8(q.cuda(), s.cuda(), 60), dy.cuda(), out=whole[:, :64])
    assert torch.equal(whole[:, :64].cpu(), torch.from_numpy(reference(q, s, 60, dy)).bfloat16())
    assert torch.isnan(whole[:, 64:]).all()


@pytest.mark.parametrize("rows,cols,outs", [(500, 600, 256), (300, 1024, 512), (9000, 512, 64)])
@pytest.mark.parametrize("first", [1, 2, 3, 16])
def test_rows_of_a_larger_checkpoint(rows, cols, outs, first):
    # scales that start on no 4- or 16-byte boundary
    q, s, dy = integers(rows + first, cols, outs, "f16", 9)
    s = s[:, :-(-cols // 32)].contiguous()
    qd, sd = q.cuda()[first:], s.cuda()[first:]
    got = tg.ckpt8_wgrad(tg.Checkpoint8(qd, sd, cols), dy[first:].cuda())
    want = torch.from_numpy(reference(q[first:], s[first:], cols, dy[first:])).half()
    assert torch.equal(got.cpu(), want)


def test_nothing_to_sum_and_nothing_to_do():
    kept = tg.Checkpoint8.empty(0, 100, "cuda")
    out = torch.full((100, 24), float("nan"), dtype=torch.float16, device="cuda")[:, :16]
    tg.ckpt8_wgrad(kept, torch.empty((0, 16), dtype=torch.float16, device="cuda"), out=out)
    assert (out == 0).all() and torch.isnan(out.as_strided((99, 8), (24, 1), 16)).all()
    kept = tg.Checkpoint8.empty(5, 0, "cuda")
    assert tg.ckpt8_wgrad(kept, torch.ones((5, 8), dtype=torch.float16, device="cuda")).shape == (0, 8)
    kept = tg.Checkpoint8.empty(5, 7, "cuda")
    assert tg.ckpt8_wgrad(kept, torch.ones((5, 0), dtype=torch.float16, device="cuda")).shape == (7, 0)


def test_offsets_past_32_bits():
    # 600000 rows of 8192 bytes: 4.9e9 bytes of q
    rows, cols, outs = 600000, 8192, 8
    q = torch.zeros((rows, cols), dtype=torch.uint8, device="cuda")
    s = torch.full((rows, cols // 32), 127, dtype=torch.uint8, device="cuda")
    at = torch.tensor([0, 262144, 524288, 599999])
    qp, sp, dyp = integers(4, cols, outs, "bf16", 2)
    q[at] = qp.cuda()
    s[at] = sp.cuda()
    dy = torch.ones((rows, outs), dtype=torch.bfloat16, device="cuda")
    dy[at] = dyp.cuda()
    got = tg.ckpt8_wgrad(tg.Checkpoint8(q, s, cols), dy)
    assert torch.equal(got.cpu(), torch.from_numpy(reference(qp, sp, cols, dyp)).bfloat16())


def test_another_stream_and_a_graph():
    q, s, dy = integers(6000, 300, 264, "f16", 4)
    kept, dyd = tg.Checkpoint8(q.cuda(), s.cuda(), 300), dy.cuda()
    want = torch.from_numpy(reference(q, s, 300, dy)).half()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tg.ckpt8_wgrad(kept, dyd, stream=side)
    side.synchronize()
    assert torch.equal(got.cpu(), want)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(got)
    with torch.cuda.graph(graph):
        tg.ckpt8_wgrad(kept, dyd, out=out)
    for scale in (1, -1, 2):
        dyd.copy_(dy * scale)
        graph.replay()
        assert torch.equal(out.cpu(), want * scale)


@pytest.mark.parametrize("cta", [0, 1])
@pytest.mark.parametrize("rows,cols,outs", [(1000, 256, 256), (9000, 60, 64)])
def test_a_missing_fill_is_reported(rows, cols, outs, cta):
    q, s, dy = integers(rows, cols, outs, "bf16", 6)
    kept, dyd = tg.Checkpoint8(q.cuda(), s.cuda(), cols), dy.cuda()
    out = torch.empty((cols, outs), dtype=torch.bfloat16, device="cuda")
    nbytes = tg.tg_ckpt8_wgrad_workspace_bytes(rows, cols, outs)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    args = (kept.q, kept.s, dyd, out, rows, cols, outs, outs, outs, "bf16", ws)
    with pytest.raises(tg.TgError) as e:
        tg.tg_ckpt8_wgrad_debug(*args, watchdog_ns=200_000_000, inject_skip_phase=(cta << 32) + 5)
    assert e.value.code == tg.TG_ERR_TIMEOUT
    tg.tg_ckpt8_wgrad_debug(*args)               # the context, TMEM and barriers are as before
    assert torch.equal(out.cpu(), torch.from_numpy(reference(q, s, cols, dy)).bfloat16())
