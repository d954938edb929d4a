"""The build without torch: the C library needs none, only the Python binding of
the operators around the products does.  Compilers are stand-ins here that write
empty outputs."""
import os
import types

import pytest

from moe_expert_gb300 import build


@pytest.fixture
def fake_tools(tmp_path, monkeypatch):
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "subprocess", types.SimpleNamespace(run=run))
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libmoex.so"))
    monkeypatch.setattr(build, "NATIVE", str(tmp_path / "_native.so"))
    return ran


def _without_torch(monkeypatch):
    find = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_without_torch_the_library_is_built(fake_tools, monkeypatch, capsys):
    _without_torch(monkeypatch)
    assert build.build() == build.LIB and os.path.exists(build.LIB) and not os.path.exists(build.NATIVE)
    assert all(c[0] == "nvcc" for c in fake_tools)
    assert "torch" in capsys.readouterr().err


def test_the_binding_follows_once_torch_is_there(fake_tools, monkeypatch):
    pytest.importorskip("torch")
    build.build()
    assert os.path.exists(build.NATIVE)
    with monkeypatch.context() as m:
        _without_torch(m)
        build.build()
        assert not os.path.exists(build.NATIVE)      # one of an older library is not left behind
    del fake_tools[:]
    build.build()
    assert os.path.exists(build.NATIVE) and any(build.BINDING in c for c in fake_tools)
