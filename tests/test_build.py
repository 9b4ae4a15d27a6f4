"""The build with stand-ins for the compilers (no GPU, nothing is compiled): libttt.so needs hipcc alone, the block
operators' binding PyTorch and g++ as well."""
import importlib.util
import os
import stat

import pytest

from test_sequence_layers_amd import build as B

OK = """#!/bin/sh
while [ $# -gt 1 ]; do [ "$1" = -o ] && echo "$0" > "$2"; shift; done
"""
BAD = "#!/bin/sh\necho no such header\nexit 1\n"


@pytest.fixture
def at(tmp_path, monkeypatch):
    """Writes the two stand-ins and points the build at them and at an empty folder."""
    def set_up(hipcc=OK, cxx=OK):
        for name, text in (("hipcc", hipcc), ("cxx", cxx)):
            if text is not None:
                (tmp_path / name).write_text(text)
                os.chmod(tmp_path / name, os.stat(tmp_path / name).st_mode | stat.S_IXUSR)
        monkeypatch.setattr(B, "HIPCC", str(tmp_path / "hipcc"))
        monkeypatch.setenv("CXX", str(tmp_path / "cxx"))
        monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path / "objects"))
        monkeypatch.setattr(B, "LIB", str(tmp_path / "libttt.so"))
        monkeypatch.setattr(B, "NATIVE", str(tmp_path / "_seq_native.so"))
        return tmp_path

    return set_up


def _no_torch(monkeypatch):
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))


def test_both_are_built(at):
    d = at()
    assert B.build() == str(d / "libttt.so")
    assert (d / "libttt.so").read_text().strip().endswith("hipcc") and (d / "_seq_native.so").read_text().strip().endswith("cxx")
    assert not list(d.glob("*.tmp"))


def test_without_pytorch_the_library_is_built_alone(at, monkeypatch, capfd):
    d = at(cxx=None)
    (d / "_seq_native.so").write_text("an older one")
    _no_torch(monkeypatch)
    assert B.build() == str(d / "libttt.so")
    assert (d / "libttt.so").exists() and not (d / "_seq_native.so").exists()
    assert "_seq_native.so" in capfd.readouterr().err


@pytest.mark.parametrize("cxx", [BAD, None])
def test_a_failing_binding_is_an_error_behind_the_library(at, cxx):
    d = at(cxx=cxx)
    (d / "_seq_native.so").write_text("an older one")
    with pytest.raises(RuntimeError, match="seq_native.cpp"):
        B.build()
    assert (d / "libttt.so").exists() and not (d / "_seq_native.so").exists() and not list(d.glob("*.tmp"))


@pytest.mark.parametrize("hipcc", [BAD, None])
def test_a_failing_source_leaves_what_was_built(at, hipcc):
    d = at(hipcc=hipcc)
    (d / "libttt.so").write_text("as it was")
    (d / "_seq_native.so").write_text("as it was")
    with pytest.raises(RuntimeError, match=r"\.hip"):
        B.build()
    assert (d / "libttt.so").read_text() == "as it was" and (d / "_seq_native.so").read_text() == "as it was"


def test_a_failing_link_leaves_what_was_built(at):
    d = at(hipcc="#!/bin/sh\ncase \"$*\" in *-shared*) echo no space; exit 1;; esac\n" + OK.split("\n", 1)[1])
    (d / "libttt.so").write_text("as it was")
    (d / "_seq_native.so").write_text("as it was")
    with pytest.raises(RuntimeError, match="link failed"):
        B.build()
    assert (d / "libttt.so").read_text() == "as it was" and (d / "_seq_native.so").read_text() == "as it was"
    assert not (d / "_seq_native.so.tmp").exists()
