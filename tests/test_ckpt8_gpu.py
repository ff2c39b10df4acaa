"""Activation checkpoints in 8 bits: pack and unpack, bit for bit against the oracle (powers of two
and single roundings leave no tolerance)."""

import numpy as np
import pytest
import torch

import persistent_warp_specialized_gb300 as tg
from gpu_helpers import ensure_library
from oracle import train

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def library():
    ensure_library()


def assert_packs(x, kept):
    q, s = train.pack(x.double().numpy())
    np.testing.assert_array_equal(kept.s.cpu().numpy(), s)
    got = kept.q.cpu().numpy()
    nan = np.isnan(train.E4M3[q])
    assert np.isnan(train.E4M3[got[nan]]).all()
    np.testing.assert_array_equal(got[~nan], q[~nan])


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 31), (2, 33), (5, 100), (64, 256),
                                       (7, 1000), (3, 2047), (300, 4096), (2, 70001)])
def test_pack_and_unpack(rows, cols, dtype):
    gen = torch.Generator().manual_seed(rows + cols)
    x = torch.randn((rows, cols), generator=gen) * torch.exp2(
        torch.randint(-12, 4, (rows, cols), generator=gen).float())
    x = x.to(DT[dtype])
    kept = tg.ckpt8_pack(x.cuda())
    assert kept.q.shape == (rows, -(-cols // 32) * 32) and kept.cols == cols
    assert_packs(x, kept)
    v = train.unpack(kept.q.cpu().numpy(), kept.s.cpu().numpy(), cols)
    for out in DT.values():
        want = torch.from_numpy(v).to(out)       # binary64 -> out, one rounding
        assert torch.equal(tg.ckpt8_unpack(kept, out).cpu(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_magnitude_and_every_tie(dtype):
    # all 2^16 bf16 patterns: zeros, subnormals, ties, infinities, NaN; neighbours in a block differ
    # by large factors in one order and hardly at all in the other
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16).view(256, 256)
    for t in (x, x.t().contiguous()):
        t = t.to(DT[dtype])
        assert_packs(t, tg.ckpt8_pack(t.cuda()))


def test_fp16_patterns():
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.float16).view(256, 256)
    for t in (x, x.t().contiguous()):
        kept = tg.ckpt8_pack(t.cuda())
        assert_packs(t, kept)
        v = train.unpack(kept.q.cpu().numpy(), kept.s.cpu().numpy(), 256)
        back = tg.ckpt8_unpack(kept, torch.float16).cpu().double().numpy()
        np.testing.assert_array_equal(back, v)   # fp16 holds what fp16 packs to


def test_unpack_takes_any_bytes():
    # every element byte under every scale byte, E4M3 NaN and scale 255 among them
    q = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(256, 1)
    s = torch.arange(256, dtype=torch.int32).to(torch.uint8)[:, None].repeat(1, 8).contiguous()
    kept = tg.Checkpoint8(q.cuda(), s.cuda(), 256)
    v = torch.from_numpy(train.unpack(q.numpy(), s.numpy(), 256))
    for out in DT.values():
        got, want = tg.ckpt8_unpack(kept, out).cpu(), v.to(out)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got[~torch.isnan(got)], want[~torch.isnan(want)])


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("offset,pad", [(0, 8), (0, 3), (1, 0), (5, 11)])
def test_row_strides_and_unaligned_bases(dtype, offset, pad):
    rows, cols = 21, 333
    gen = torch.Generator().manual_seed(offset)
    x = torch.randn((rows, cols), generator=gen).to(DT[dtype])
    flat = torch.full((offset + rows * (cols + pad),), float("nan"), dtype=x.dtype, device="cuda")
    view = flat[offset:].view(rows, cols + pad)[:, :cols]
    view.copy_(x)
    kept = tg.ckpt8_pack(view)
    assert_packs(x, kept)
    view.fill_(float("nan"))
    tg.ckpt8_unpack(kept, x.dtype, out=view)
    v = train.unpack(kept.q.cpu().numpy(), kept.s.cpu().numpy(), cols)
    assert torch.equal(view.cpu(), torch.from_numpy(v).to(x.dtype))
    if pad:
        assert torch.isnan(flat[offset:].view(rows, cols + pad)[:, cols:]).all()


def test_nothing_to_do():
    for shape in ((0, 64), (4, 0)):
        kept = tg.ckpt8_pack(torch.empty(shape, dtype=torch.float16, device="cuda"))
        assert tg.ckpt8_unpack(kept, torch.float32).shape == shape


def test_a_checkpoint_is_an_operand_of_the_mxfp8_product():
    # x^ W^ by tg_gemm_mxfp8 on the checkpoints themselves: their scales are packed as they are
    from persistent_warp_specialized_gb300 import workloads

    M, N, K = 200, 136, 256
    gen = torch.Generator().manual_seed(1)
    x, w = torch.randn((M, K), generator=gen), torch.randn((N, K), generator=gen)
    kx, kw = tg.ckpt8_pack(x.cuda()), tg.ckpt8_pack(w.cuda())
    for t, k in ((x, kx), (w, kw)):              # the recipe of the MXFP8 workloads
        q, s = workloads._mx_quantize(t)
        assert torch.equal(k.q.cpu(), q) and torch.equal(k.s.cpu(), s)
    c = tg.mxfp8_gemm(kx.q, kx.s, kw.q, kw.s)
    a = train.unpack(kx.q.cpu().numpy(), kx.s.cpu().numpy(), K)
    b = train.unpack(kw.q.cpu().numpy(), kw.s.cpu().numpy(), K)
    # K products summed in fp32 (truncating adds: 2^-23 each), one rounding to bf16
    tol = K * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T) + 2.0 ** -8 * np.abs(a @ b.T) + 2.0 ** -134
    assert (np.abs(c.cpu().double().numpy() - a @ b.T) <= tol).all()
