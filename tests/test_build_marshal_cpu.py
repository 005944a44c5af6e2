"""The host binding is rebuilt for another torch or Python, and refused before it is loaded."""
import os
import subprocess

import pytest

from decodability_aware_token_b200 import _abi, build


@pytest.fixture
def place(tmp_path, monkeypatch):
    so, stamp = str(tmp_path / "_marshal.so"), str(tmp_path / "_marshal.abi")
    for mod, names in ((_abi, ("MARSHAL_PATH", "MARSHAL_STAMP")), (build, ("MARSHAL", "STAMP"))):
        monkeypatch.setattr(mod, names[0], so)
        monkeypatch.setattr(mod, names[1], stamp)
    monkeypatch.setattr(_abi, "_marshal", None)
    runs = []

    def compiler(cmd, **kw):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(build.subprocess, "run", compiler)
    return so, stamp, runs


def test_a_binding_for_another_torch_or_python_is_rebuilt(place, monkeypatch):
    so, stamp, runs = place
    build.build_marshal()
    build.build_marshal()
    assert len(runs) == 1 and _abi.marshal_stamp() == _abi.marshal_abi()
    now = _abi.marshal_abi()
    monkeypatch.setattr(_abi, "marshal_abi", lambda: now.replace("torch ", "torch 9"))
    build.build_marshal()                                   # newer than its sources, but for another torch
    build.build_marshal()
    assert len(runs) == 2 and _abi.marshal_stamp() == _abi.marshal_abi() != now
    os.remove(stamp)
    build.build_marshal()                                   # not known what it was built for
    assert len(runs) == 3
    build.build_marshal(force=True)
    assert len(runs) == 4


def test_a_binding_for_another_python_is_refused_before_it_is_loaded(place, monkeypatch):
    so, stamp, _ = place
    with pytest.raises(ImportError, match="missing"):
        _abi.load_marshal()
    build.build_marshal()
    monkeypatch.setattr(_abi.importlib.util, "spec_from_file_location", lambda *a: pytest.fail("loaded"))
    with open(stamp, "w") as f:
        f.write("torch 1.0, cxx11 abi 0, cpython-36m\n")
    with pytest.raises(ImportError, match="rebuild"):
        _abi.load_marshal()


def test_the_built_binding_is_this_torchs():
    assert _abi.marshal_stamp() in (None, _abi.marshal_abi())
