"""How the library and the module of the binding's compiled calls are built and
put in place (no GPU), on sources of a few lines."""
import glob
import importlib.machinery
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


def test_modules_of_other_interpreters_do_not_stay(tree):
    for name in ("_calls.so", "_calls.cpython-39-x86_64-linux-gnu.so"):
        (tree / name).write_text("before")
    b.build()
    assert _left(tree) == sorted(map(os.path.basename, (b.LIB, b.CALLS)))
    assert b.CALLS.endswith(importlib.machinery.EXTENSION_SUFFIXES[0]) and "cpython" in b.CALLS


_ENTRIES = ("mds_status_string", "mds_last_error", "mds_qk_norm_rope", "mds_qk_norm_rope_append",
            "mds_paged_attention_sinks", "mds_lm_head_mxfp4")


@pytest.mark.parametrize("abi,torch_version,error", [
    (0, None, None), (1, None, "interface"), (0, "2.1.0", "torch"), (0, "", "torch"), (0, "{}0", "torch"),
    (0, "{}+other", None)])
def test_the_module_refuses_another_library_or_torch(tmp_path, abi, torch_version, error):
    # the real module beside a library that has its entry points and some version
    import torch
    import markov_draft_sampling_amd as mds
    if not os.path.exists(b.CALLS):
        b.build()
    version = mds.abi_version() + abi
    (tmp_path / "lib.cpp").write_text("".join(f'extern "C" int {n}() {{ return 0; }}\n' for n in _ENTRIES)
                                      + f'extern "C" int mds_abi_version() {{ return {version}; }}\n')
    cxx = shutil.which("g++") or os.path.join(os.path.dirname(os.path.realpath(b._hipcc())), "amdclang++")
    subprocess.run([cxx, "-shared", "-fPIC", "-o", str(tmp_path / "libmds.so"), str(tmp_path / "lib.cpp")], check=True)
    shutil.copy(b.CALLS, tmp_path)
    code = f"import sys, torch; sys.path.insert(0, {str(tmp_path)!r})\n"
    if torch_version is not None:
        code += f"torch.__version__ = {torch_version.format(torch.__version__.split('+')[0])!r}\n"
    r = subprocess.run([sys.executable, "-c", code + "import _calls"], capture_output=True, text=True)
    if error is None:
        assert r.returncode == 0, r.stderr
    else:
        assert r.returncode != 0 and "ImportError: built" in r.stderr and error in r.stderr.splitlines()[-1], r.stderr
