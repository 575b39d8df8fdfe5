"""The build without a GPU and without running the real compilers: what it needs, what it rebuilds."""
import os
import stat

import pytest

from weight_only_int4_act_b200 import _build


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """_build with an empty output folder and, for nvcc, a script that writes its -o file; returns the folder."""
    script = tmp_path / "nvcc"
    script.write_text('#!/bin/sh\nwhile [ "$1" != "-o" ]; do shift; done\necho built > "$2"\n')
    script.chmod(script.stat().st_mode | stat.S_IXUSR)
    out = tmp_path / "lib"
    monkeypatch.setattr(_build, "LIB_DIR", str(out))
    monkeypatch.setattr(_build, "nvcc", lambda: str(script))
    return out


def test_library_needs_nvcc_alone(sandbox, monkeypatch):
    """Without torch (or its CUDA headers) there is no calls' module, and the library is built as ever."""
    def no_torch(out):
        raise ImportError("No module named 'torch'")
    monkeypatch.setattr(_build, "calls_command", no_torch)
    with pytest.warns(UserWarning, match="torch"):
        path = _build.build(variants=tuple(_build.VARIANTS))
    assert path == _build.lib_path() == os.path.join(str(sandbox), "libawq_b200.so")
    assert sorted(os.listdir(sandbox)) == ["libawq_b200.so", "libawq_b200_check.so"]


def test_failed_calls_module_leaves_the_library_in_place(sandbox, monkeypatch):
    monkeypatch.setattr(_build, "calls_command", lambda out: ["false"])
    with pytest.raises(RuntimeError, match="false failed"):
        _build.build()
    assert os.listdir(sandbox) == ["libawq_b200.so"]


def test_calls_module_is_rebuilt_for_another_torch(sandbox, monkeypatch):
    made = []

    def command(out):
        made.append(out)
        return [_build.nvcc(), "-o", out]
    monkeypatch.setattr(_build, "calls_command", command)
    _build.build()
    _build.build()
    assert len(made) == 1
    first = _build.calls_path()
    monkeypatch.setattr(_build, "torch_version", lambda: "99.0.0+cu999")
    assert _build.calls_path() != first
    _build.build()
    assert len(made) == 2 and os.path.exists(_build.calls_path())


def test_torch_version_is_the_installed_one():
    import torch
    assert _build.torch_version() == torch.__version__
