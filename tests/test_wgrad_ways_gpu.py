"""Every way through the weight gradient's kernel, bit for bit on integers: products and partial sums are
integers below 2^24.  wgrad_shapes.py says which way a shape takes."""

import pytest
import torch

import persistent_warp_specialized_gb300 as tg
from gpu_helpers import ensure_library
from test_ckpt8_wgrad_gpu import DT, integers, reference, run
from wgrad_shapes import PAIRS, WAYS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    ensure_library()


def test_the_ways_are_this_devices():
    assert tg.tg_gemm_launch_shape(8192, 8192, 8192, "pair")["workers"] == PAIRS


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", WAYS)
def test_integers_bit_exact(shape, dtype):
    q, s, dy = integers(*shape, dtype, sum(shape))
    want = torch.from_numpy(reference(q, s, shape[1], dy)).to(DT[dtype])
    got = run(q, s, shape[1], dy)
    assert torch.equal(got.cpu(), want)
    if shape[1] % 512 == 0:                      # the same scales, off the 16-byte grid: not by TMA
        sd = torch.empty(s.numel() + 4, dtype=torch.uint8, device="cuda")[4:].view(s.shape)
        sd.copy_(s)
        again = tg.ckpt8_wgrad(tg.Checkpoint8(q.cuda(), sd, shape[1]), dy.cuda())
        assert torch.equal(again, got)


@pytest.mark.parametrize("shape", [(1000, 4864, 4096), (520, 3000, 4608), (16000, 2000, 1000)])
def test_repeated_calls_give_the_same_bits(shape):
    gen = torch.Generator().manual_seed(1)
    kept = tg.ckpt8_pack(torch.randn((shape[0], shape[1]), generator=gen).cuda())
    dy = torch.randn((shape[0], shape[2]), generator=gen).bfloat16().cuda()
    first = tg.ckpt8_wgrad(kept, dy)
    assert torch.isfinite(first).all()
    assert all(torch.equal(tg.ckpt8_wgrad(kept, dy), first) for _ in range(5))


# Tiles of two N-halves: a fill missing in a pair's first unit, in its second, and in a range.
@pytest.mark.parametrize("cta", [0, 1])
@pytest.mark.parametrize("shape,phase", [((700, 2500, 2304), 5), ((1000, 4864, 4096), 20),
                                         ((16000, 2000, 1000), 7)])
def test_a_missing_fill_is_reported(shape, phase, cta):
    rows, cols, outs = shape
    q, s, dy = integers(rows, cols, outs, "bf16", 6)
    kept, dyd = tg.Checkpoint8(q.cuda(), s.cuda(), cols), dy.cuda()
    out = torch.empty((cols, outs), dtype=torch.bfloat16, device="cuda")
    nbytes = tg.tg_ckpt8_wgrad_workspace_bytes(rows, cols, outs)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    args = (kept.q, kept.s, dyd, out, rows, cols, outs, outs, outs, "bf16", ws)
    with pytest.raises(tg.TgError) as e:
        tg.tg_ckpt8_wgrad_debug(*args, watchdog_ns=200_000_000,
                                inject_skip_phase=(cta << 32) + phase)
    assert e.value.code == tg.TG_ERR_TIMEOUT
    tg.tg_ckpt8_wgrad_debug(*args)               # the context, TMEM and barriers are as before
    assert torch.equal(out.cpu(), torch.from_numpy(reference(q, s, cols, dy)).bfloat16())
