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
