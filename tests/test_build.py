"""The build's own logic, on the host: the library does not depend on the quick binding, and a
binding made for something else is neither kept nor used."""
import os
import subprocess
import sys
import warnings

import pytest
import torch

from exact_io_aware_60_b200 import build as B
from exact_io_aware_60_b200 import fa


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


def test_the_binding_is_built_again_for_another_torch(monkeypatch, tmp_path):
    """As for another Python, other flags or a newer header; not for nothing."""
    ran = []

    def compiler(cmd, **_):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_fa_binding.so"))
    monkeypatch.setattr(B, "BINDING_STAMP", str(tmp_path / "_fa_binding.stamp"), raising=False)
    monkeypatch.setattr(B.subprocess, "run", compiler)
    for change, times in ((None, 1), (None, 1), ("torch", 2), (None, 2), ("header", 3), (None, 3)):
        if change == "torch":
            monkeypatch.setattr(torch, "__version__", "9.9.9")
        elif change == "header":
            (tmp_path / "fa.h").write_text("")
            os.utime(tmp_path / "fa.h", (2 ** 32, 2 ** 32))
            monkeypatch.setattr(B, "INCLUDE", str(tmp_path))
        elif times == 3:
            os.utime(B.BINDING, (2 ** 32, 2 ** 32))
        B.build_binding()
        assert len(ran) == times


def test_a_binding_for_another_torch_is_not_used(monkeypatch):
    assert fa._quick is not None
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert fa._load_quick() is fa._quick
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    with pytest.warns(RuntimeWarning, match="9.9.9"):
        assert fa._load_quick() is None


def test_a_binding_that_cannot_be_imported_is_said(monkeypatch, tmp_path):
    monkeypatch.setitem(sys.modules, "exact_io_aware_60_b200._fa_binding", None)
    monkeypatch.delattr(sys.modules["exact_io_aware_60_b200"], "_fa_binding", raising=False)
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert fa._load_quick() is None
    monkeypatch.setattr(fa, "_HERE", str(tmp_path))   # there is none: not a word
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert fa._load_quick() is None


def test_the_binding_takes_its_signatures_from_the_header():
    with open(B.BINDING_SRC) as f:
        src = f.read()
    for name in ("fa_rope", "fa_kv_append", "fa_fwd_paged"):
        assert f"decltype(&{name})" in src
