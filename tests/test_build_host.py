"""The build of the serving calls' binding, which the rest of the package does
not need."""
import sys

import pytest

from bwd_step_b200 import build


@pytest.fixture
def binding(tmp_path, monkeypatch):
    monkeypatch.setattr(build, "SERVING", str(tmp_path / "_serving.so"))
    return tmp_path / "_serving.so"


def test_the_library_is_built_where_torch_is_absent(binding, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB
    assert not binding.exists()
    assert "PyTorch" in capsys.readouterr().err


def test_the_library_is_built_where_no_host_compiler_is(binding, monkeypatch, capsys):
    pytest.importorskip("torch")
    which = build.shutil.which
    monkeypatch.setattr(build.shutil, "which", lambda name: None if name == "g++" else which(name))
    assert build.build() == build.LIB
    assert not binding.exists()
    assert "g++" in capsys.readouterr().err
