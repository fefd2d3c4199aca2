"""When the compiled Python binding is built: not without torch, and anew when
torch or Python changed."""
import importlib.metadata
import sys

import pytest

from exact_softmax_attention_04_b200 import build_lib


@pytest.fixture
def here(tmp_path, monkeypatch):
    """The library is there and up to date, the binding is to be tmp_path's."""
    monkeypatch.setattr(build_lib, "BIND", str(tmp_path / "attn_bind.so"))
    monkeypatch.setattr(build_lib, "stale", lambda: False)
    return tmp_path


def test_the_library_is_built_without_torch(here, monkeypatch, capsys):
    def missing(name):
        raise importlib.metadata.PackageNotFoundError(name)

    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    monkeypatch.setattr(importlib.metadata, "version", missing)
    assert build_lib.build() == build_lib.LIB
    assert not (here / "attn_bind.so").exists()
    assert "torch" in capsys.readouterr().err


def test_the_binding_is_stale_after_a_change_of_torch(here, monkeypatch):
    calls = []

    def compile_(cmd):
        calls.append(cmd)
        (here / cmd[cmd.index("-o") + 1]).write_bytes(b"")

    monkeypatch.setattr(build_lib.subprocess, "check_call", compile_)
    build_lib.build()
    build_lib.build()
    assert len(calls) == 1
    installed = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: installed(name) + ".other")
    assert build_lib.bind_stale()
    build_lib.build()
    assert len(calls) == 2 and not build_lib.bind_stale()
    monkeypatch.setattr(build_lib.sysconfig, "get_config_var", lambda name: "other-python")
    assert build_lib.bind_stale()
