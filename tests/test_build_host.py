"""How the library and the binding's compiled checks are built: the library
without torch, the checks for the torch that is there."""
import os
import sys
import types

import pytest

import variable_size_all_gb300 as a2av
from variable_size_all_gb300 import _build


def test_the_library_builds_without_torch(monkeypatch):
    a2av.build()
    monkeypatch.setitem(sys.modules, "torch", None)  # (what an import of it raises without one)
    with pytest.raises(ImportError):
        import torch  # noqa: F401
    assert _build.start_marshal(force=True) is None
    assert _build.build() == _build.LIBRARY


@pytest.fixture
def place(monkeypatch, tmp_path):
    """A module and its record in a folder of their own, and the commands that would compile it."""
    import torch
    started = []

    class Process:
        code = 0

        def __init__(self, command):
            started.append(command)

        def wait(self):
            if self.code == 0:
                open(started[-1][started[-1].index("-o") + 1], "w").close()
            return self.code

    monkeypatch.setattr(_build, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(_build, "MARSHAL_TORCH", str(tmp_path / "_marshal.torch"))
    monkeypatch.setattr(_build.subprocess, "Popen", Process)
    monkeypatch.setattr(_build.shutil, "which", lambda name: "/usr/bin/" + name)
    monkeypatch.setattr(_build.os.path, "exists", lambda p: p.endswith("Python.h") or os.access(p, os.F_OK))
    return types.SimpleNamespace(torch=torch, started=started, process=Process)


def test_the_checks_are_built_for_the_torch_that_is_there(place, monkeypatch):
    _build.finish_marshal(_build.start_marshal())
    assert len(place.started) == 1 and os.path.exists(_build.MARSHAL)
    assert f'-DA2AV_TORCH="{place.torch.__version__}"' in place.started[0]
    assert _build.start_marshal() is None  # (up to date)
    monkeypatch.setattr(place.torch, "__version__", "0.0.1")
    _build.finish_marshal(_build.start_marshal())
    assert len(place.started) == 2 and '-DA2AV_TORCH="0.0.1"' in place.started[1]
    assert _build.start_marshal() is None
    os.remove(_build.MARSHAL_TORCH)  # (of a torch that nothing tells)
    assert _build.start_marshal() is not None


def test_checks_that_do_not_compile_leave_none_behind(place):
    _build.finish_marshal(_build.start_marshal())
    place.process.code = 1
    _build.finish_marshal(_build.start_marshal(force=True))
    assert not os.path.exists(_build.MARSHAL)


def test_checks_of_another_torch_are_not_used(monkeypatch):
    torch = pytest.importorskip("torch")
    for version, used in (("0.0.1", False), (torch.__version__, True)):
        module = types.SimpleNamespace(torch_version=version)
        monkeypatch.setattr(a2av, "_marshal", module, raising=False)
        assert (a2av._load_marshal() is module) == used
        assert used or a2av._load_marshal() is a2av._PlainMarshal
