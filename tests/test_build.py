"""How the library and the module of the binding's compiled calls are built and
put in place (no GPU), on sources of a few lines."""
import glob
import os
import shutil
import subprocess
import sys

import pytest

from markov_draft_sampling_amd import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package's tree with an earlier build in place."""
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "lib.hip").write_text('extern "C" int answer() { return 42; }\n')
    (tmp_path / "csrc" / "calls.cpp").write_text('#include <Python.h>\nextern "C" int answer();\n'
                                                 'extern "C" int asked() { return answer(); }\n')
    monkeypatch.setattr(b, "HERE", str(tmp_path))
    monkeypatch.setattr(b, "CSRC", str(tmp_path / "csrc"))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libmds.so"))
    monkeypatch.setattr(b, "CALLS", str(tmp_path / os.path.basename(b.CALLS)))
    monkeypatch.setattr(b, "SOURCES", ("lib.hip",))
    for path in (b.LIB, b.CALLS):
        with open(path, "w") as f:
            f.write("before")
    return tmp_path


def _old(path):
    with open(path, "rb") as f:
        return f.read() == b"before"


def _left(tree):
    return sorted(os.path.basename(p) for p in glob.glob(str(tree / "*.so*")))


@pytest.mark.parametrize("gxx", [True, False])
def test_both_are_put_in_place(tree, monkeypatch, gxx):
    if not gxx:
        which = shutil.which
        monkeypatch.setattr(b.shutil, "which", lambda name: None if name == "g++" else which(name))
    assert b.build() == b.LIB
    assert not _old(b.LIB) and not _old(b.CALLS)
    assert _left(tree) == sorted(map(os.path.basename, (b.LIB, b.CALLS)))
    # it finds the library beside it, by its final name (in a process of its own: this one may have loaded the real ones)
    code = f"import ctypes, torch; assert ctypes.CDLL({b.CALLS!r}).asked() == 42"
    subprocess.run([sys.executable, "-c", code], check=True)


@pytest.mark.parametrize("source", ["lib.hip", "calls.cpp"])
def test_nothing_is_put_in_place_when_one_fails(tree, source):
    (tree / "csrc" / source).write_text("this is no program\n")
    with pytest.raises(RuntimeError, match="failed"):
        b.build()
    assert _old(b.LIB) and _old(b.CALLS)
    assert _left(tree) == sorted(map(os.path.basename, (b.LIB, b.CALLS)))


def test_the_library_alone_without_torch(tree, monkeypatch, capsys):
    find = b.importlib.util.find_spec
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None if name == "torch" else find(name))
    assert b.build() == b.LIB
    assert not _old(b.LIB) and _left(tree) == ["libmds.so"]  # no module of an earlier library stays
    assert "torch is not installed" in capsys.readouterr().err
