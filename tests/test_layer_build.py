"""The library is built and linked whatever becomes of the marshalling module, which alone needs torch (the commands are
recorded, not run)."""
import builtins
import os

import pytest

from selective_state_space_22_amd import build as lib_build


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """The commands of a build whose outputs go to tmp_path; a command whose output is in `failing` raises."""
    ran, failing = [], set()

    def run(cmd, verbose):
        out = cmd[cmd.index("-o") + 1]
        if out in failing:
            raise RuntimeError(f"{cmd[0]} failed")
        ran.append(out)
        open(out, "w").close()

    for name, leaf in (("LIB", "lib.so"), ("BIND", "_bind.so"), ("OBJ_DIR", "obj")):
        monkeypatch.setattr(lib_build, name, str(tmp_path / leaf))
    monkeypatch.setattr(lib_build, "hipcc", lambda: "hipcc")
    monkeypatch.setattr(lib_build, "_run", run)
    return ran, failing


def test_library_and_module(commands):
    pytest.importorskip("torch")
    assert lib_build.build() == lib_build.LIB
    assert os.path.exists(lib_build.LIB) and os.path.exists(lib_build.BIND)
    assert len(commands[0]) == len(lib_build.SOURCES) + 2


def test_library_without_torch(commands, monkeypatch, capsys):
    real = builtins.__import__

    def no_torch(name, *args, **kw):
        if name == "torch" or name.startswith("torch."):
            raise ModuleNotFoundError("No module named 'torch'")
        return real(name, *args, **kw)

    monkeypatch.setattr(builtins, "__import__", no_torch)
    assert lib_build.build() == lib_build.LIB
    assert os.path.exists(lib_build.LIB) and not os.path.exists(lib_build.BIND)
    assert "No module named 'torch'" in capsys.readouterr().err


def test_library_where_the_module_does_not_compile(commands):
    pytest.importorskip("torch")
    commands[1].add(lib_build.BIND + ".tmp")
    with pytest.raises(RuntimeError, match="lib.so is built, _bind.so is not"):
        lib_build.build()
    assert os.path.exists(lib_build.LIB) and not os.path.exists(lib_build.BIND)


def test_a_source_that_does_not_compile_ends_the_build(commands):
    commands[1].add(os.path.join(lib_build.OBJ_DIR, "conv.o"))
    with pytest.raises(RuntimeError, match="hipcc failed"):
        lib_build.build()
    assert not os.path.exists(lib_build.LIB)
