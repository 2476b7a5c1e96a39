"""What build() makes and in which order, with the compilers replaced by stand-ins that write empty files; CPU."""
import importlib.util
import os

import pytest

from exact_attention_72_gb300 import build


@pytest.fixture
def made(monkeypatch, tmp_path):
    """A package folder of its own; the names of what was compiled and linked, in order."""
    log = []

    def compile_one(nvcc, src, verbose):
        log.append(os.path.basename(src))
        return src

    def run(cmd, what):
        log.append(what)
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(build, "PKG_DIR", str(tmp_path))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / build.LIB_NAME))
    monkeypatch.setattr(build, "CALLS_PATH", str(tmp_path / os.path.basename(build.CALLS_PATH)))
    if hasattr(build, "CALLS_STAMP"):
        monkeypatch.setattr(build, "CALLS_STAMP", str(tmp_path / "_build" / "calls.txt"))
    monkeypatch.setattr(build, "_compile", compile_one)
    monkeypatch.setattr(build, "_run", run)
    return log


def test_library_and_calls(made):
    assert build.build() == build.LIB_PATH and os.path.exists(build.LIB_PATH) and os.path.exists(build.CALLS_PATH)
    n = len(made)
    assert build.up_to_date() and build.build() and len(made) == n       # nothing to do
    os.utime(build.CALLS_PATH, (0, 0))
    assert not build.up_to_date()
    build.build()
    assert len(made) == n + 2 and "link" not in made[n:]                 # the calls alone
    os.utime(build.LIB_PATH, (0, 0))
    build.build()
    assert made[n + 2:].count("link") == 1 and not any("calls" in x for x in made[n + 2:])


def test_the_library_needs_no_torch(made, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build(force=True) == build.LIB_PATH and os.path.exists(build.LIB_PATH)
    assert not os.path.exists(build.CALLS_PATH) and not any("calls" in x for x in made)
    assert build.up_to_date() and build.build() == build.LIB_PATH


def test_a_failing_compilation_of_the_calls_leaves_the_library(made, monkeypatch):
    run = build._run

    def failing(cmd, what):
        if "calls.cpp" in what:
            raise RuntimeError(what + " failed")
        run(cmd, what)
    monkeypatch.setattr(build, "_run", failing)
    with pytest.raises(RuntimeError, match="calls.cpp failed"):
        build.build()
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.CALLS_PATH)


def test_the_calls_are_made_for_one_python_and_one_torch(made, monkeypatch, tmp_path):
    """Another torch counts whatever the age of its files, another interpreter by its ABI, and neither's module is loaded."""
    from exact_attention_72_gb300 import binding
    assert os.path.basename(build.CALLS_PATH) == "_calls" + build.EXT_SUFFIX
    assert not build.calls_fit()                       # nothing built yet
    build.build()
    assert build.calls_fit() and build.up_to_date()
    torch = tmp_path / "other" / "torch"
    torch.mkdir(parents=True)
    (torch / "version.py").write_text("__version__ = '0'\n")
    os.utime(torch / "version.py", (0, 0))             # older than the module
    with monkeypatch.context() as m:
        m.setattr(build, "_torch_dir", lambda: str(torch))
        assert not build.calls_fit() and not build.up_to_date()
        m.setattr(binding, "_CALLS", None)
        m.setattr(binding, "lib", lambda: None)
        with pytest.raises(RuntimeError, match="another Python or torch"):
            binding._calls()
    assert build.up_to_date()
    monkeypatch.setattr(build, "EXT_SUFFIX", ".cpython-399-other.so")
    assert not build.calls_fit()
