"""Where the calls' binding cannot be compiled or loaded, the library is built and the calls go on in Python (no GPU needed)."""
import os
import subprocess
import types

import pytest

import call_stubs as C
import quantized_moe_expert_routed_gb300 as M

B = M._build


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The library and the binding in another folder, and compilers of the test's own: (what ran, which programs fail)."""
    ran, failing = [], set()

    def run(cmd, **kw):
        ran.append(os.path.basename(cmd[0]))
        if ran[-1] in failing:
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    M.load()  # (the true one, before its path changes)
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(B, "calls_path", lambda: str(tmp_path / "calls.so"))
    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setenv("CXX", "g++")
    return ran, failing


def test_the_library_is_built_without_the_binding(elsewhere):
    ran, failing = elsewhere
    failing.add("g++")
    assert B.build() == B.LIB and os.path.exists(B.LIB) and not os.path.exists(B.calls_path())
    assert ran.count("g++") == 1 and ran.count("nvcc") == len(B.SOURCES) + 1
    assert "no such header" in open(B.calls_failed()).read()
    B.build()  # neither is tried again
    assert len(ran) == len(B.SOURCES) + 2
    failing.clear()
    os.utime(B.calls_failed(), (0, 0))  # the sources are newer
    B.build()
    assert ran.count("g++") == 2 and os.path.exists(B.calls_path()) and ran.count("nvcc") == len(B.SOURCES) + 1


def test_no_host_compiler_at_all(elsewhere, monkeypatch):
    def run(cmd, **kw):
        raise FileNotFoundError(cmd[0])
    open(B.LIB, "w").close()
    monkeypatch.setattr(subprocess, "run", run)
    assert B.build() == B.LIB and "not compiled" in open(B.calls_failed()).read()


def test_a_binding_of_older_sources_goes(elsewhere):
    ran, failing = elsewhere
    failing.add("g++")
    for f in (B.LIB, B.calls_path()):
        open(f, "w").close()
    os.utime(B.calls_path(), (0, 0))
    B.build()
    assert ran == ["g++"] and not os.path.exists(B.calls_path())


def test_a_failing_library_is_an_error(elsewhere):
    ran, failing = elsewhere
    failing.add("nvcc")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        B.build()


@pytest.mark.parametrize("there", [False, True])
def test_calls_go_on_in_python_and_say_so_once(there, monkeypatch, tmp_path):
    lib = C.install(monkeypatch)
    monkeypatch.setattr(M, "_calls", None)
    monkeypatch.setattr(B, "calls_path", lambda: str(tmp_path / "calls.so"))
    with open(B.calls_path() if there else B.calls_failed(), "w") as f:
        f.write("no such header")  # (there: a file that is no library)
    with pytest.warns(RuntimeWarning, match="go through Python") as said:
        for name in C.CALLS * 2:
            tensors, rest = C.arguments(name)
            getattr(M, name)(**tensors, **rest)
    assert len(said) == 1 and [c[0] for c in lib.calls] == C.CALLS * 2
    assert there or "no such header" in str(said[0].message)
