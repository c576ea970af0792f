"""What a build installs, and when: with stand-ins for the compilers, in a directory of its own."""
import os
import stat
import sysconfig

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


def commands(sandbox):
    log = sandbox / "log"
    lines = log.read_text().splitlines() if log.exists() else []
    log.write_text("")
    return len(lines)


def test_the_module_is_built_again_for_another_torch(sandbox, monkeypatch):
    """A file of the same age serves the Python and torch that it was compiled against alone."""
    fa_build.build()
    assert commands(sandbox) == 3 and fa_build.up_to_date()  # a.cu, the link, calls.cpp
    fa_build.build()
    assert commands(sandbox) == 0
    monkeypatch.setattr(fa_build, "built_for", lambda: "another")
    assert fa_build.library_up_to_date() and not fa_build.up_to_date()
    fa_build.build()
    assert commands(sandbox) == 1 and fa_build.up_to_date()
    os.remove(fa_build.LIB_PATH)
    fa_build.build()
    assert commands(sandbox) == 2 and fa_build.up_to_date()
    os.utime(fa_build.CALLS_SOURCE, (2 ** 32, 2 ** 32))
    assert not fa_build.up_to_date()


def test_an_unfinished_build_is_not_up_to_date(sandbox, monkeypatch):
    fa_build.build()
    os.utime(fa_build.CALLS_SOURCE, (2 ** 32, 2 ** 32))
    monkeypatch.setattr(fa_build, "calls_command", lambda out: ["false", out])
    with pytest.raises(RuntimeError, match="calls.cpp"):
        fa_build.build()
    assert not fa_build.up_to_date()


def test_the_module_tells_what_it_was_built_for(monkeypatch):
    import tiled_exact_attention_forward_b200 as fa

    fa_build.build()
    assert fa._compiled().built_for == fa_build.built_for()
    assert sysconfig.get_config_var("EXT_SUFFIX") in fa._compiled().__file__
    monkeypatch.setattr(fa, "_COMPILED", None)
    monkeypatch.setattr(fa_build, "built_for", lambda: "another")
    with pytest.raises(ImportError, match="another Python or torch"):
        fa._compiled()
