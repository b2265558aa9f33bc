"""What the build does when a compiler fails or torch changes, with compilers that only write their output files."""
import os
import subprocess
import types

import pytest


@pytest.fixture
def build(monkeypatch, tmp_path):
    """The build in folders of its own; .ran: the outputs of the commands in their order, .failing: parts of outputs that fail."""
    from rotation_int4_w4a4_b200 import build as b
    monkeypatch.setattr(b, "OBJDIR", str(tmp_path / "obj"))
    monkeypatch.setattr(b, "LIBDIR", str(tmp_path / "lib"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib" / "libpq.so"))
    monkeypatch.setattr(b, "CALL_LIB", str(tmp_path / "lib" / os.path.basename(b.CALL_LIB)))
    state = types.SimpleNamespace(ran=[], failing={}, lib=tmp_path / "lib", module=b, call=b.CALL_LIB)

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        state.ran.append(os.path.basename(out))
        for part, how in state.failing.items():
            if part in out:
                if isinstance(how, BaseException):
                    raise how
                return subprocess.CompletedProcess(cmd, how, "", "no such header")
        open(out, "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", run)
    return state


def test_everything_once(build):
    assert build.module.build() == str(build.lib / "libpq.so")
    made = sorted(os.listdir(build.lib))
    assert made == sorted(["libpq.so", os.path.basename(build.call)])
    build.ran.clear()
    build.module.build()
    assert build.ran == []


@pytest.mark.parametrize("how", [1, FileNotFoundError("g++")], ids=["fails", "missing"])
def test_the_library_needs_no_module(build, capsys, how):
    """A torch without CUDA, a Python without headers, no C++ compiler: the library is linked, and what is missing is said."""
    build.failing = {"_pqcall": how}
    assert build.module.build() == str(build.lib / "libpq.so")
    assert os.listdir(build.lib) == ["libpq.so"]
    assert "_pqcall" in capsys.readouterr().err
    build.failing = {}
    build.ran.clear()
    build.module.build()
    assert build.ran == [os.path.basename(build.call)]     # tried again


def test_a_module_that_fails_leaves_no_old_one(build):
    """One of an older header would call the new library by its old signatures."""
    build.module.build()
    os.utime(build.module.CALL_LIB, (0, 0))
    build.failing = {"_pqcall": 1}
    build.module.build()
    assert os.listdir(build.lib) == ["libpq.so"]


@pytest.mark.parametrize("part", ["fp4.cu.o", "libpq.so"])
def test_the_library_itself_must_build(build, part):
    build.failing = {part: 1}
    with pytest.raises(RuntimeError):
        build.module.build()
    assert not (build.lib / "libpq.so").exists()


def test_without_torch(build, monkeypatch, capsys):
    build.module.build()
    os.utime(build.module.CALL_LIB, (0, 0))
    monkeypatch.setattr(build.module.importlib.util, "find_spec", lambda name: None)
    assert build.module.build() and os.listdir(build.lib) == ["libpq.so"] and "torch is not installed" in capsys.readouterr().err


def test_another_torch_or_python_has_another_module(monkeypatch, tmp_path):
    """The module reads torch's C++ objects in place: one built for another torch is not loaded, whatever its file's age."""
    import sysconfig
    from rotation_int4_w4a4_b200 import build as b
    import torch
    assert os.path.basename(b.CALL_LIB) == b.call_lib_name(torch.version.__version__)
    assert b.CALL_LIB.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    (tmp_path / "version.py").write_text("from typing import Optional\n__version__ = '9.8.7+cu999'\ncuda = None\n")
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: types.SimpleNamespace(submodule_search_locations=[str(tmp_path)]))
    assert b.torch_version() == "9.8.7+cu999"
    assert b.call_lib_name("9.8.7+cu999") != b.call_lib_name(torch.version.__version__)


def test_modules_of_other_sources_are_removed(build):
    """Those for other torches too: they would be loaded again when that torch comes back, against the new library."""
    build.module.build()
    for name, when in (("_pqcall-1.0.so", 0), ("_pqcall.so", 0), ("_pqcall-2.0.so", None)):
        (build.lib / name).touch()
        if when is not None:
            os.utime(build.lib / name, (when, when))
    build.module.build()
    assert sorted(os.listdir(build.lib)) == sorted(["libpq.so", os.path.basename(build.call), "_pqcall-2.0.so"])


def test_a_module_of_another_torch_is_not_loaded(monkeypatch):
    from rotation_int4_w4a4_b200 import build as b
    b.build()
    from rotation_int4_w4a4_b200 import pq
    import torch
    monkeypatch.setattr(pq, "_call", None)
    assert pq._caller() is not pq._NoModule
    monkeypatch.setattr(torch.version, "__version__", "9.8.7+cu999")
    with pytest.warns(RuntimeWarning, match="9.8.7"):
        assert pq._caller() is pq._NoModule
