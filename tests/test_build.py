"""What build() compiles and when, with the compilers replaced by a recorder:
the library does not depend on what only the Python binding needs."""
import os
import subprocess

import pytest

from block_sparse_flash_gb300 import build as b


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """Compilers that only write their output file; `broken`: names of those
    that fail.  Returns (calls, broken): one name per call."""
    calls, broken = [], set()

    def run(cmd, **_):
        name = os.path.basename(cmd[0])
        calls.append(name)
        if name in broken:
            if "missing" in broken:
                raise FileNotFoundError(cmd[0])
            return subprocess.CompletedProcess(cmd, 1, "", "Python.h: No such file or directory")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libsplash.so"))
    monkeypatch.setattr(b.subprocess, "run", run)
    return calls, broken


def test_everything_once_and_then_nothing(tools):
    calls, _ = tools
    assert b.build() == b.LIB
    assert calls.count("nvcc") == len(b.SOURCES) + 1 and calls.count("g++") == 2
    assert os.path.exists(b.LIB) and os.path.exists(b.binding_path())
    del calls[:]
    b.build()
    assert calls == []


@pytest.mark.parametrize("how", [{"g++"}, {"g++", "missing"}])
def test_the_library_is_built_without_what_the_binding_needs(tools, how):
    calls, broken = tools
    broken |= how
    with pytest.warns(RuntimeWarning, match="serving calls"):
        assert b.build() == b.LIB
    assert os.path.exists(b.LIB) and not os.path.exists(b.binding_path())
    broken.clear()
    del calls[:]
    b.build()
    assert calls == ["g++", "g++"] and os.path.exists(b.binding_path())


def test_another_torch_needs_another_binding_only(tools, monkeypatch):
    calls, _ = tools
    b.build()
    del calls[:]
    other = os.path.join(b.OUT_DIR, "_binding.another.so")
    monkeypatch.setattr(b, "binding_path", lambda: other)
    b.build()
    assert calls == ["g++", "g++"] and os.path.exists(other)


def test_a_binding_that_no_longer_builds_is_not_left_behind(tools):
    """An old binding would pass argument structs of another layout."""
    calls, broken = tools
    b.build()
    os.utime(b.binding_path(), (0, 0))
    broken.add("g++")
    with pytest.warns(RuntimeWarning):
        b.build()
    assert not os.path.exists(b.binding_path()) and "nvcc" not in calls[len(b.SOURCES) + 3:]


def test_a_library_that_does_not_build_is_an_error(tools):
    _, broken = tools
    broken.add("nvcc")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        b.build()
