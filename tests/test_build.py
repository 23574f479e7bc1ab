"""The build script: the library needs hipcc alone, also where the Python extension cannot be built."""
import os
import sys

import pytest

from swiglu_mlp_amd import build


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """The build with outputs in tmp_path and a compiler that writes its -o file."""
    cc = tmp_path / "cc"
    cc.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\necho built > "$2"\n')
    cc.chmod(0o755)
    monkeypatch.setattr(build, "HIPCC", str(cc))
    monkeypatch.setattr(build, "ROOT", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "marshal.so"))
    return tmp_path


def test_library_without_torch(fake, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)      # import torch fails
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.MARSHAL)
    assert "torch" in capsys.readouterr().out


def test_library_is_there_where_the_extension_fails(fake, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setenv("PATH", str(fake))                # no g++
    with pytest.raises((RuntimeError, OSError)):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.MARSHAL)
