"""The compiled checks of tensor arguments read torch's objects: they are rebuilt for another torch,
and those of another torch are refused before they read anything."""
import os
import sysconfig
import types

import pytest

import speculative_decoding_draft_04_gb300 as package
from speculative_decoding_draft_04_gb300 import _lib, build

pytest.importorskip("torch")


def test_a_build_for_another_torch_is_stale(tmp_path, monkeypatch):
    build.build()
    assert not build.is_stale()
    other = tmp_path / "args_for.txt"
    other.write_text("torch 1.0.0 0000")
    monkeypatch.setattr(build, "ARGS_FOR", str(other))
    assert build.is_stale()
    monkeypatch.setattr(build, "ARGS_FOR", str(tmp_path / "none.txt"))
    assert build.is_stale()


def test_the_file_is_named_for_its_python():
    assert os.path.basename(build.ARGS) == "_args" + sysconfig.get_config_var("EXT_SUFFIX")
    build.build()
    _lib._types()
    assert _lib._args.__file__ == build.ARGS and _lib._args.built_for == build.built_for()


def test_checks_of_another_torch_are_refused(monkeypatch):
    def use(error):
        raise AssertionError("called")
    fake = types.SimpleNamespace(built_for="torch 1.0.0 0000", use=use)
    monkeypatch.setattr(package, "_args", fake, raising=False)
    monkeypatch.setattr(_lib, "_torch", None)
    with pytest.raises(_lib.SpecError, match="torch 1.0.0"):
        _lib._types()
    assert _lib._torch is None
