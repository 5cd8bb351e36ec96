"""The build on machines that lack what only the Python binding needs: the library is built all the
same.  Compilers are stand-ins that write an empty file."""
import os

import pytest

from kda_chunked_recurrent_b200 import build as b


@pytest.fixture
def machine(tmp_path, monkeypatch):
    """Targets in a folder of their own, and the commands that were run."""
    ran = []

    def run(cmd, check):
        assert check
        ran.append(os.path.basename(cmd[0]))
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "BIND", str(tmp_path / "bind.so"))
    monkeypatch.setattr(b, "nvcc_path", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(b.subprocess, "run", run)
    return ran


def _lack(what, monkeypatch):
    if what == "torch":
        real = b.importlib.util.find_spec
        monkeypatch.setattr(b.importlib.util, "find_spec",
                            lambda n: None if n == "torch" else real(n))
        monkeypatch.setitem(__import__("sys").modules, "torch", None)
    elif what == "g++":
        real_which = b.shutil.which
        monkeypatch.setattr(b.shutil, "which", lambda n: None if n == "g++" else real_which(n))
    else:
        monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": "/nowhere"})


@pytest.mark.parametrize("what", ["torch", "g++", "Python.h"])
@pytest.mark.parametrize("force", [False, True])
def test_the_library_is_built_without_what_the_binding_needs(machine, monkeypatch, capsys, what, force):
    _lack(what, monkeypatch)
    assert b.needs_build()
    assert b.build(force=force) == b.LIB
    assert machine == ["nvcc"] and os.path.exists(b.LIB) and not os.path.exists(b.BIND)
    assert what in capsys.readouterr().err
    assert not b.needs_build()


def test_both_are_built_where_all_is_there(machine, capsys):
    b.build()
    assert machine == ["nvcc", "g++"] and os.path.exists(b.BIND) and not b.needs_build()
    assert capsys.readouterr().err == ""


def test_a_failing_compiler_is_an_error(machine, monkeypatch):
    def run(cmd, check):
        raise b.subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(b.subprocess, "run", run)
    with pytest.raises(b.subprocess.CalledProcessError):
        b.build()
