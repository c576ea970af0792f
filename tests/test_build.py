"""What a build installs, and when: with stand-ins for the compilers, in a directory of its own."""
import os
import stat

import pytest

from tiled_exact_attention_forward_b200 import build as fa_build


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """One source, and a compiler that writes its output file and notes its command."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    for name in ("a.cu", "calls.cpp"):
        (csrc / name).write_text("")
    cc = tmp_path / "cc"
    cc.write_text(f'#!/bin/sh\necho "$@" >> {tmp_path}/log\n'
                  'while [ "$1" != "-o" ]; do shift; done\necho built > "$2"\n')
    cc.chmod(cc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(fa_build, "CSRC", str(csrc))
    monkeypatch.setattr(fa_build, "ROOT", str(tmp_path))
    monkeypatch.setattr(fa_build, "OBJ_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(fa_build, "LIB_PATH", str(tmp_path / "libfa_b200.so"))
    monkeypatch.setattr(fa_build, "CALLS_PATH", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(fa_build, "CALLS_SOURCE", str(csrc / "calls.cpp"))
    monkeypatch.setattr(fa_build, "nvcc", lambda: str(cc))
    monkeypatch.setattr(fa_build, "calls_command", lambda out: [str(cc), "-o", out])
    return tmp_path


def test_the_library_is_installed_without_the_module(sandbox, monkeypatch):
    monkeypatch.setattr(fa_build, "calls_command", lambda out: ["false", out])
    with pytest.raises(RuntimeError, match="calls.cpp"):
        fa_build.build()
    assert os.path.exists(fa_build.LIB_PATH) and not os.path.exists(fa_build.CALLS_PATH)
