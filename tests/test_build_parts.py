"""The library is built where the module for torch tensors cannot be: a compiler that refuses it, one that is not
there, a torch without the libraries it links.  nvcc and g++ are stand-ins that write what they are asked for."""

import os
import stat

import pytest

import persistent_warp_specialized_gb300 as tg
from persistent_warp_specialized_gb300 import _build

WRITES = """#!/bin/sh
echo "$@" >> "{log}"
while [ $# -gt 0 ]; do
  case "$1" in
    -o) echo made > "$2"; shift;;
    {refused}) echo "no such thing: $1" >&2; exit 1;;
  esac
  shift
done
"""


def script(path, log, refused="nothing"):
    path.write_text(WRITES.format(log=log, refused=refused))
    path.chmod(path.stat().st_mode | stat.S_IXUSR)


@pytest.fixture()
def place(tmp_path, monkeypatch):
    """Everything the build writes goes to tmp_path; returns it, with the stand-ins in its bin."""
    build_dir = tmp_path / "_build"
    for name, value in {"BUILD_DIR": build_dir, "LIB_PATH": tmp_path / "libtg.so",
                        "STAMP": build_dir / "libtg.stamp", "TORCH_PATH": tmp_path / "tg_torch.so",
                        "TORCH_STAMP": build_dir / "tg_torch.stamp",
                        "TORCH_ERROR": build_dir / "tg_torch.error"}.items():
        monkeypatch.setattr(_build, name, str(value), raising=False)
    (tmp_path / "bin").mkdir()
    script(tmp_path / "bin" / "nvcc", tmp_path / "nvcc.log")
    script(tmp_path / "bin" / "g++", tmp_path / "gxx.log")
    monkeypatch.setenv("NVCC", str(tmp_path / "bin" / "nvcc"))
    monkeypatch.setenv("PATH", f"{tmp_path}/bin:/usr/bin:/bin")
    return tmp_path


def calls(log):
    return len(log.read_text().splitlines()) if log.exists() else 0


def test_both_are_built_once(place):
    assert _build.build() == str(place / "libtg.so")
    assert (place / "tg_torch.so").exists() and _build.torch_error() is None
    before = calls(place / "nvcc.log"), calls(place / "gxx.log")
    _build.build()
    assert before == (calls(place / "nvcc.log"), calls(place / "gxx.log")) and min(before) > 0
    os.remove(place / "tg_torch.so")            # the one does not take the other along
    _build.build()
    assert (place / "tg_torch.so").exists() and calls(place / "nvcc.log") == before[0]


@pytest.mark.parametrize("refused", ["*tg_torch.cpp", "-lc10_cuda"])
def test_the_library_without_the_module(place, refused, monkeypatch, capsys):
    script(place / "bin" / "g++", place / "gxx.log", refused)
    (place / "tg_torch.so").write_text("one of other sources")
    _build.build()
    assert (place / "libtg.so").exists() and not (place / "tg_torch.so").exists()
    assert "no such thing" in _build.torch_error() and "no such thing" in capsys.readouterr().err
    # not again while nothing changed
    before = calls(place / "gxx.log")
    _build.build()
    assert calls(place / "gxx.log") == before
    # the reason is what a call that needs the module says
    monkeypatch.setattr(tg, "TORCH_PATH", _build.TORCH_PATH)
    monkeypatch.setattr(tg, "_torch_calls", None)
    monkeypatch.setattr(tg, "_lib", object())
    with pytest.raises(RuntimeError, match="no such thing"):
        tg.input_grad(None, None)
    # and by force, once it can be built
    script(place / "bin" / "g++", place / "gxx.log")
    _build.build(force=True)
    assert (place / "tg_torch.so").exists() and _build.torch_error() is None


def test_no_compiler_for_the_module(place, monkeypatch):
    os.remove(place / "bin" / "g++")
    monkeypatch.setattr(_build.shutil, "which", lambda name: None)
    monkeypatch.setenv("PATH", f"{place}/bin")
    # a stand-in for nvcc that needs nothing on PATH
    (place / "bin" / "nvcc").write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do [ "$1" = -o ] && echo made > "$2"; shift; done\n')
    _build.build()
    assert (place / "libtg.so").exists() and "g++" in _build.torch_error()


def test_a_library_that_cannot_be_built_raises(place):
    script(place / "bin" / "nvcc", place / "nvcc.log", "*tg_train.cu")
    with pytest.raises(RuntimeError, match="(?s)nvcc failed.*no such thing"):
        _build.build()
    assert not (place / "libtg.so").exists()
