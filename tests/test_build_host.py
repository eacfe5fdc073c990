"""The build of the serving calls' binding, which the rest of the package does
not need, and which depends on the PyTorch and Python that it was built for."""
import sys
import sysconfig
import types

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


def _runs(binding, monkeypatch):
    """The compiler's calls while the binding is asked for, each of which makes the file."""
    made = []

    def run(cmd, **kw):
        made.append(cmd)
        binding.write_bytes(b"\x7fELF")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(build.subprocess, "run", run)
    return made


@pytest.mark.parametrize("what", ["torch", "python"])
def test_the_binding_is_rebuilt_for_another_torch_or_python(binding, monkeypatch, what):
    torch = pytest.importorskip("torch")
    made = _runs(binding, monkeypatch)
    build._build_serving(False, False)
    build._build_serving(False, False)
    assert len(made) == 1  # up to date
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "0.0.1")
    else:
        monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-999")
    build._build_serving(False, False)
    build._build_serving(False, False)
    assert len(made) == 2


def test_a_binding_of_unknown_make_is_rebuilt(binding, monkeypatch):
    pytest.importorskip("torch")
    binding.write_bytes(b"\x7fELF")
    made = _runs(binding, monkeypatch)
    build._build_serving(False, False)
    assert len(made) == 1
