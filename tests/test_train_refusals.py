"""What the training operators refuse, and with which error.  No GPU: every case returns before any
CUDA call, or from the Python layer."""

import pytest
import torch

import persistent_warp_specialized_gb300 as tg
from persistent_warp_specialized_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def library():
    _build.build()
    tg.load_library()


def refused(code, call, *args, **kw):
    with pytest.raises(tg.TgError) as e:
        call(*args, stream=0, **kw)
    assert e.value.code == code, e.value


# x, gamma, beta, y, mean, rstd, yq, ys, rows, cols, ld_x, ld_y, dtype
FWD = [256, 512, 512, 1024, 0, 0, None, None, 4, 32, 32, 32, "bf16"]


@pytest.mark.parametrize("code,at,value", [
    (tg.TG_ERR_ARG, 12, 7), (tg.TG_ERR_ARG, 8, -1), (tg.TG_ERR_ARG, 9, -1),
    (tg.TG_ERR_ARG, 8, 1 << 31), (tg.TG_ERR_ARG, 9, 1 << 31), (tg.TG_ERR_ARG, 10, 31),
    (tg.TG_ERR_ARG, 11, 31), (tg.TG_ERR_ARG, 0, None), (tg.TG_ERR_ALIGN, 0, 257),
    (tg.TG_ERR_ARG, 6, 4096)])
def test_layer_norm_forward(code, at, value):
    args = list(FWD)
    args[at] = value
    refused(code, tg.tg_layernorm_fwd, *args)


def test_layer_norm_forward_options():
    refused(tg.TG_ERR_ARG, tg.tg_layernorm_fwd, *FWD, eps=-1.0)
    refused(tg.TG_ERR_ARG, tg.tg_layernorm_fwd, *FWD, eps=float("nan"))
    refused(tg.TG_ERR_ARG, tg.tg_layernorm_fwd, *FWD, param_dtype="f16")   # values are bf16
    args = FWD[:8] + [0, 32, 32, 32, "bf16"]
    assert tg.tg_layernorm_fwd(*args, stream=0) == 0
    args = FWD[:8] + [4, 0, 32, 32, "bf16"]
    assert tg.tg_layernorm_fwd(*args, stream=0) == 0


# dy, x, xq, xs, gamma, mean, rstd, dx, dgamma, dbeta, rows, cols, ld_dy, ld_x, ld_dx, dtype
BWD = [256, 512, None, None, None, 1024, 1024, 2048, None, None, 4, 32, 32, 32, 32, "f16"]


@pytest.mark.parametrize("code,at,value", [
    (tg.TG_ERR_ARG, 15, -3), (tg.TG_ERR_ARG, 10, -1), (tg.TG_ERR_ARG, 11, 1 << 31),
    (tg.TG_ERR_ARG, 12, 31), (tg.TG_ERR_ARG, 13, 31), (tg.TG_ERR_ARG, 14, 31),
    (tg.TG_ERR_ARG, 0, None), (tg.TG_ERR_ALIGN, 0, 257), (tg.TG_ERR_ARG, 2, 4096),
    (tg.TG_ERR_ARG, 3, 4096)])
def test_layer_norm_backward(code, at, value):
    args = list(BWD)
    args[at] = value
    refused(code, tg.tg_layernorm_bwd, *args)


def test_layer_norm_backward_options():
    both = list(BWD)
    both[2], both[3] = 4096, 8192
    refused(tg.TG_ERR_ARG, tg.tg_layernorm_bwd, *both)
    refused(tg.TG_ERR_ARG, tg.tg_layernorm_bwd, *BWD, param_dtype="bf16")
    refused(tg.TG_ERR_ARG, tg.tg_layernorm_bwd, *BWD, workspace=4096, workspace_bytes=-1)
    for args in ((-1, 8), (8, 1 << 31)):
        with pytest.raises(tg.TgError):
            tg.tg_layernorm_bwd_workspace_bytes(*args)
    assert tg.tg_layernorm_bwd_workspace_bytes(0, 8) == 0


@pytest.mark.parametrize("call", [tg.tg_ckpt8_pack, tg.tg_ckpt8_unpack])
def test_checkpoints(call):
    def args(**kw):
        a = dict(a=256, b=512, c=1024, rows=4, cols=40, ld=40, dtype="bf16") | kw
        return [a[k] for k in ("a", "b", "c", "rows", "cols", "ld", "dtype")]

    refused(tg.TG_ERR_ARG, call, *args(dtype=9))
    refused(tg.TG_ERR_ARG, call, *args(rows=-1))
    refused(tg.TG_ERR_ARG, call, *args(cols=1 << 31))
    refused(tg.TG_ERR_ARG, call, *args(ld=39))
    refused(tg.TG_ERR_ARG, call, *args(a=None))
    refused(tg.TG_ERR_ALIGN, call, *args(a=257))
    assert call(*args(rows=0), stream=0) == 0
    assert call(*args(cols=0), stream=0) == 0


def test_python_layer():
    x = torch.zeros((4, 40), dtype=torch.float16)
    with pytest.raises(ValueError):
        tg.Checkpoint8(torch.zeros((4, 40), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8), 40)
    with pytest.raises(TypeError):
        tg.Checkpoint8(torch.zeros((4, 64)), torch.zeros((4, 2)), 40)
    with pytest.raises(ValueError):
        tg.Checkpoint8(torch.zeros((64, 4), dtype=torch.uint8).t(), torch.zeros((4, 2), dtype=torch.uint8), 40)
    with pytest.raises(TypeError):
        tg.ckpt8_pack(x.double())
    with pytest.raises(ValueError):
        tg.ckpt8_pack(x.t())                                 # strided along its rows
    with pytest.raises(ValueError):
        tg.ckpt8_pack(x[:1].expand(4, 40))                   # overlapping rows
    with pytest.raises(ValueError):
        tg.layer_norm(x, torch.zeros(39))
    with pytest.raises(TypeError):
        tg.layer_norm(x, torch.zeros(40), torch.zeros(40, dtype=torch.float16))
    with pytest.raises(TypeError):
        tg.layer_norm(x, torch.zeros(40, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        tg.layer_norm(x, out=torch.zeros((4, 41), dtype=torch.float16))
    stat = torch.zeros(4)
    with pytest.raises(ValueError):
        tg.layer_norm_backward(x, x[:3], stat, stat)
    with pytest.raises(ValueError):
        tg.layer_norm_backward(x, x, stat.half(), stat)
    kept = tg.Checkpoint8.empty(4, 72, "cpu")
    with pytest.raises(ValueError):
        tg.layer_norm_backward(x, kept, stat, stat)
    with pytest.raises(ValueError):
        tg.ckpt8_unpack(kept, torch.float16, out=x)


# q, s, dY, dW, rows, cols, outs, ld_dy, ld_dw, dtype
WGRAD = [256, 512, 1024, 2048, 16, 40, 64, 64, 64, "bf16"]


@pytest.mark.parametrize("code,at,value", [
    (tg.TG_ERR_ARG, 9, "f32"), (tg.TG_ERR_ARG, 9, 5), (tg.TG_ERR_ARG, 4, -1),
    (tg.TG_ERR_ARG, 5, 1 << 31), (tg.TG_ERR_ARG, 6, -8), (tg.TG_ERR_ALIGN, 6, 60),
    (tg.TG_ERR_ARG, 7, 56), (tg.TG_ERR_ALIGN, 7, 68), (tg.TG_ERR_ARG, 8, 56),
    (tg.TG_ERR_ALIGN, 8, 66), (tg.TG_ERR_ARG, 3, None), (tg.TG_ERR_ALIGN, 3, 2056)])
def test_weight_gradient(code, at, value):
    args = list(WGRAD)
    args[at] = value
    refused(code, tg.tg_ckpt8_wgrad, *args)


def test_weight_gradient_sizes():
    for args in ((-1, 8, 8), (8, -1, 8), (8, 8, 1 << 31), (8, 1 << 31, 8), (8, 8, 12),
                 (8, (1 << 31) - 1, (1 << 31) - 8)):
        with pytest.raises(tg.TgError):
            tg.tg_ckpt8_wgrad_workspace_bytes(*args)
    assert tg.tg_ckpt8_wgrad_workspace_bytes(0, 8, 8) == 0
    refused(tg.TG_ERR_ARG, tg.tg_ckpt8_wgrad, *WGRAD, workspace=4096, workspace_bytes=-1)
    assert tg.tg_ckpt8_wgrad(*WGRAD[:5], 0, *WGRAD[6:], stream=0) == 0
    kept = tg.Checkpoint8.empty(4, 72, "cpu")
    with pytest.raises(ValueError):
        tg.ckpt8_wgrad(kept, torch.zeros((5, 8), dtype=torch.float16))
    with pytest.raises(ValueError):
        tg.ckpt8_wgrad(kept, torch.zeros((4, 8), dtype=torch.float16),
                       out=torch.zeros((72, 16), dtype=torch.float16))
