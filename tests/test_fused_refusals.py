"""What the input gradient, the gated projections and the cross entropy refuse, and with which error.  No GPU:
every case returns before any CUDA call, or from the Python layer."""

import pytest
import torch

import persistent_warp_specialized_gb300 as tg
from persistent_warp_specialized_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def library():
    _build.build()
    tg.load_library()


def call(fn, names, defaults, **kw):
    a = dict(defaults) | kw
    extra = {k: a.pop(k) for k in ("workspace", "workspace_bytes") if k in a}
    return fn(*[a[n] for n in names], stream=0, **extra)


def refused(code, fn, names, defaults, **kw):
    with pytest.raises(tg.TgError) as e:
        call(fn, names, defaults, **kw)
    assert e.value.code == code, e.value
    return str(e.value)


GRAD = ["dY", "W", "dX", "rows", "cols", "outs", "ld_dy", "ld_w", "ld_dx", "dtype"]
GRAD_OK = dict(dY=256, W=512, dX=1024, rows=4, cols=32, outs=64, ld_dy=64, ld_w=64, ld_dx=32,
               dtype="bf16")
FWD = ["x", "wg", "wu", "h", "g", "u", "rows", "cols", "outs", "ld_x", "ld_wg", "ld_wu", "ld_h",
       "ld_g", "ld_u", "act", "dtype"]
FWD_OK = dict(x=256, wg=512, wu=1024, h=2048, g=None, u=None, rows=4, cols=32, outs=64, ld_x=32,
              ld_wg=64, ld_wu=64, ld_h=64, ld_g=64, ld_u=64, act="silu", dtype="f16")
BWD = ["dh", "g", "u", "x", "wg", "wu", "dx", "dwg", "dwu", "rows", "cols", "outs", "ld_dh", "ld_g",
       "ld_u", "ld_x", "ld_wg", "ld_wu", "ld_dx", "ld_dwg", "ld_dwu", "act", "dtype"]
BWD_OK = dict(dh=256, g=512, u=768, x=1024, wg=1280, wu=1536, dx=2048, dwg=4096, dwu=8192, rows=4,
              cols=32, outs=64, ld_dh=64, ld_g=64, ld_u=64, ld_x=32, ld_wg=64, ld_wu=64, ld_dx=32,
              ld_dwg=64, ld_dwu=64, act="gelu", dtype="bf16")
XF = ["x", "w", "targets", "loss", "lse", "rows", "cols", "vocab", "ld_x", "ld_w", "ignore", "dtype"]
XF_OK = dict(x=256, w=512, targets=1024, loss=2048, lse=4096, rows=4, cols=32, vocab=7, ld_x=32,
             ld_w=32, ignore=-100, dtype="bf16")
XB = ["dloss", "x", "w", "targets", "lse", "dx", "dw", "rows", "cols", "vocab", "ld_x", "ld_w",
      "ld_dx", "ld_dw", "ignore", "dtype"]
XB_OK = dict(dloss=128, x=256, w=512, targets=1024, lse=4096, dx=8192, dw=16384, rows=4, cols=32,
             vocab=7, ld_x=32, ld_w=32, ld_dx=32, ld_dw=32, ignore=-100, dtype="f16")
ALL = {"input_grad": (tg.tg_input_grad, GRAD, GRAD_OK), "gated_fwd": (tg.tg_gated_fwd, FWD, FWD_OK),
       "gated_bwd": (tg.tg_gated_bwd, BWD, BWD_OK), "xent_fwd": (tg.tg_xent_fwd, XF, XF_OK),
       "xent_bwd": (tg.tg_xent_bwd, XB, XB_OK)}


@pytest.mark.parametrize("name", ALL)
def test_types_and_sizes(name):
    fn, names, ok = ALL[name]
    for bad in (2, 7, -1):                                  # float32 is for the norm
        refused(tg.TG_ERR_ARG, fn, names, ok, dtype=bad)
    wide = "vocab" if "vocab" in ok else "outs"
    for size in ("rows", "cols", wide):
        for bad in (-8, 1 << 31):
            refused(tg.TG_ERR_ARG, fn, names, ok, **{size: bad})
    odd = dict(cols=36) | {k: 40 for k in names if k.startswith("ld_")}
    refused(tg.TG_ERR_ALIGN, fn, names, dict(ok) | {wide: 24}, **odd)
    refused(tg.TG_ERR_ARG, fn, names, ok, workspace=4096, workspace_bytes=-1)


@pytest.mark.parametrize("name", ALL)
def test_strides(name):
    fn, names, ok = ALL[name]
    extra = dict(g=1 << 16, u=1 << 17) if name == "gated_fwd" else {}
    for ld in [n for n in names if n.startswith("ld_")]:
        refused(tg.TG_ERR_ARG, fn, names, ok, **extra, **{ld: 24})
        refused(tg.TG_ERR_ARG, fn, names, ok, **extra, **{ld: 1 << 31})
        refused(tg.TG_ERR_ALIGN, fn, names, ok, **extra, **{ld: 68})


@pytest.mark.parametrize("name,out", [("input_grad", "dX"), ("gated_fwd", "h"), ("gated_bwd", "dx"),
                                      ("xent_fwd", "loss"), ("xent_bwd", "dx")])
def test_the_first_output_must_be_there_and_aligned(name, out):
    fn, names, ok = ALL[name]
    if name not in ("gated_bwd", "xent_bwd"):               # there it may be left out
        refused(tg.TG_ERR_ARG, fn, names, ok, **{out: None})
    refused(tg.TG_ERR_ALIGN, fn, names, ok, **{out: ok[out] + 2})
    refused(tg.TG_ERR_ARG, fn, names, ok)                   # not a device pointer


def test_choices():
    for act in (2, -1):
        refused(tg.TG_ERR_ARG, *ALL["gated_fwd"], act=act)
        refused(tg.TG_ERR_ARG, *ALL["gated_bwd"], act=act)
    refused(tg.TG_ERR_ARG, *ALL["gated_fwd"], g=4096)       # without u
    refused(tg.TG_ERR_ARG, *ALL["gated_bwd"], dwu=None)
    for fn in ("xent_fwd", "xent_bwd"):
        refused(tg.TG_ERR_ARG, *ALL[fn], vocab=0)
        refused(tg.TG_ERR_ARG, *ALL[fn], cols=0)
    with pytest.raises(ValueError, match="silu"):
        call(*ALL["gated_fwd"], act="relu")


def test_too_many_tiles():
    big = (1 << 31) - 8
    lds = {"ld_dy": big, "ld_w": big, "ld_dx": big}
    refused(tg.TG_ERR_ARG, *ALL["input_grad"], rows=big, cols=big, outs=8, **lds)
    refused(tg.TG_ERR_ARG, *ALL["xent_fwd"], rows=big, vocab=big)


def test_nothing_to_do():
    assert call(*ALL["input_grad"], rows=0) == 0
    assert call(*ALL["input_grad"], cols=0) == 0
    assert call(*ALL["gated_fwd"], rows=0) == 0
    assert call(*ALL["gated_fwd"], outs=0) == 0
    assert call(*ALL["gated_bwd"], cols=0) == 0
    assert call(*ALL["gated_bwd"], dx=None, dwg=None, dwu=None) == 0
    assert call(*ALL["xent_fwd"], rows=0) == 0
    assert call(*ALL["xent_bwd"], dx=None, dw=None) == 0


def test_workspace_sizes():
    for fn in (tg.tg_input_grad_workspace_bytes, tg.tg_gated_fwd_workspace_bytes,
               tg.tg_gated_bwd_workspace_bytes, tg.tg_xent_bwd_workspace_bytes):
        assert fn(0, 32, 64) == 0
        for sizes in ((-1, 32, 64), (4, 36, 64), (4, 32, 1 << 31)):
            with pytest.raises(tg.TgError):
                fn(*sizes)
    assert tg.tg_xent_fwd_workspace_bytes(0, 32, 7) == 0


def test_python_layer():
    x = torch.zeros((4, 32), dtype=torch.bfloat16)
    w = torch.zeros((32, 64), dtype=torch.bfloat16)
    e = torch.zeros((7, 32), dtype=torch.bfloat16)
    dh = torch.zeros((4, 64), dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)
    for call_ in (lambda: tg.gated_forward(x.float(), w, w), lambda: tg.gated_forward(x, w.half(), w),
                  lambda: tg.input_grad(dh.float(), w), lambda: tg.input_grad(dh, w.half()),
                  lambda: tg.linear_cross_entropy(x, e.half(), t)):
        with pytest.raises(TypeError):
            call_()
    for call_ in (lambda: tg.gated_forward(x, w, w[:, :32]), lambda: tg.gated_forward(x, w.t(), w.t()),
                  lambda: tg.gated_forward(x[0], w, w), lambda: tg.gated_forward(x, w, w, act="tanh"),
                  lambda: tg.gated_forward(x, w, w, out=x),
                  lambda: tg.gated_backward(dh, dh, dh[:2], x, w, w),
                  lambda: tg.gated_backward(dh, dh, dh, x[:3], w, w),
                  lambda: tg.input_grad(x, w), lambda: tg.input_grad(dh, w, out=dh),
                  lambda: tg.linear_cross_entropy(x, e, t.int()),
                  lambda: tg.linear_cross_entropy(x, e, t[:3]),
                  lambda: tg.linear_cross_entropy(x, e[:, :24], t),
                  lambda: tg.linear_cross_entropy_backward(f.double(), x, e, t, f),
                  lambda: tg.linear_cross_entropy_backward(f, x, e, t, f[:2])):
        with pytest.raises(ValueError):
            call_()
