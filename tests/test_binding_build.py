"""The extension of the expert operators is rebuilt for, and refused under, another PyTorch, Python
or set of flags than it was built for."""
from __future__ import annotations

import os
import shutil

import pytest
import torch

import w8a8_int8_quantized_sq_b200 as sq
from w8a8_int8_quantized_sq_b200 import build as sq_build


@pytest.fixture()
def built(tmp_path, monkeypatch):
    """A copy of the built extension that counts as the one of the package; the list of the
    compiler's runs, which only copy it again."""
    sq_build.build()
    for end in ("", ".key"):
        if os.path.exists(sq_build.BINDING + end):
            shutil.copy2(sq_build.BINDING + end, tmp_path / ("_binding.so" + end))
    real = sq_build.BINDING
    runs = []

    def run(cmd, what, verbose):
        runs.append(cmd)
        shutil.copy2(real, cmd[cmd.index("-o") + 1])

    monkeypatch.setattr(sq_build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(sq_build, "_run", run)
    monkeypatch.setattr(sq, "_ext", None)
    return runs


def other_torch(monkeypatch):
    monkeypatch.setattr(torch, "__version__", "9.9.9+cu0")


def other_python(monkeypatch):
    real = sq_build.sysconfig.get_config_var
    monkeypatch.setattr(sq_build.sysconfig, "get_config_var",
                        lambda name: "cpython-399" if name == "SOABI" else real(name))


def other_flags(monkeypatch):
    monkeypatch.setattr(sq_build, "BINDING_FLAGS", ["-O0"], raising=False)


def test_unchanged_is_kept(built):
    sq_build.build_binding()
    assert not built
    assert sq._extension() is not None


@pytest.mark.parametrize("change", [other_torch, other_python, other_flags])
def test_a_change_rebuilds_and_is_refused_until_then(built, monkeypatch, change):
    change(monkeypatch)
    with pytest.raises(RuntimeError, match="build it with"):
        sq._extension()
    sq_build.build_binding()
    assert len(built) == 1
    sq_build.build_binding()
    assert len(built) == 1  # once


def test_a_file_that_does_not_say_is_refused(built, monkeypatch):
    sq._extension()
    monkeypatch.setattr(sq, "_ext", None)
    from w8a8_int8_quantized_sq_b200 import _binding
    monkeypatch.delattr(_binding, "built_for")
    with pytest.raises(RuntimeError, match="unknown.*build it with"):
        sq._extension()


def test_a_missing_key_rebuilds(built):
    os.remove(sq_build.BINDING + ".key")
    sq_build.build_binding()
    assert len(built) == 1
