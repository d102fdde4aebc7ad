"""The build's own logic, on the host: the library does not depend on the quick binding."""
import subprocess

import pytest

from exact_io_aware_60_b200 import build as B


@pytest.mark.parametrize("what", [RuntimeError("g++ failed"), ImportError("no torch"), FileNotFoundError("g++")])
def test_the_library_is_built_whatever_becomes_of_the_binding(what, monkeypatch, capsys):
    done = []

    def no_binding(*_):
        raise what

    monkeypatch.setattr(B, "build_library", lambda *a: done.append(a) or B.LIB, raising=False)
    monkeypatch.setattr(B, "up_to_date", lambda: bool(done.append("up to date") or True))
    monkeypatch.setattr(B, "build_binding", no_binding)
    assert B.build() == B.LIB
    assert done
    assert str(what) in capsys.readouterr().err


def test_a_library_that_does_not_compile_is_an_error(monkeypatch, tmp_path):
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libfa.so"))
    monkeypatch.setattr(B, "build_binding", lambda *_: None)
    monkeypatch.setattr(B.subprocess, "run",
                        lambda *a, **k: subprocess.CompletedProcess(a, 1, "", "error"))
    with pytest.raises(RuntimeError):
        B.build()
