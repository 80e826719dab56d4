"""The serving operators where the module of the compiled calls is not built
(no GPU): attention is called all the same, the others say what is missing."""
import os
import shutil
import subprocess
import sys

import pytest

import markov_draft_sampling_amd as mds
from markov_draft_sampling_amd import _serving


def test_a_package_without_the_module(tmp_path):
    here = os.path.dirname(os.path.abspath(mds.__file__))
    package = tmp_path / os.path.basename(here)
    package.mkdir()
    for name in ("__init__.py", "_serving.py", "build.py"):
        shutil.copy(os.path.join(here, name), package)
    os.symlink(mds.library_path(), package / "libmds.so")
    code = """
import torch, markov_draft_sampling_amd as mds
from markov_draft_sampling_amd import _serving
assert mds.abi_version() == 2 and _serving._calls(needed=False) is None
_serving.importlib.util.find_spec = None  # (looked for once)
assert _serving._calls(needed=False) is None
x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
for call in (lambda: mds.qk_norm_rope(x, x, x, None, x, x), lambda: mds.lm_head_mxfp4(x[0], x, x, x, 1)):
    try:
        call()
    except mds.MdsError as e:
        assert "compiled calls" in str(e) and "markov_draft_sampling_amd.build" in str(e), e
    else:
        raise AssertionError
try:
    mds.paged_attention(x, x, x, x, x, x, x, 1, 1)
except mds.MdsError as e:
    assert "GPU" in str(e), e
else:
    raise AssertionError
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env={**os.environ, "PYTHONPATH": str(tmp_path)},
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def _args(**kw):
    import torch
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    i32 = torch.int32
    a = dict(q=z(3, 4, 64), k_pages=z(8, 16, 2, 64), v_pages=z(8, 16, 2, 64), block_table=z(2, 4, t=i32),
             query_start=z(3, t=i32), seq_lens=z(2, t=i32), out=z(3, 4, 64), max_q_len=2, max_seq_len=64, scale=None,
             causal=True, window=16, sinks=4, idx_map=None, k_scale=None, v_scale=None, lse=z(3, 4, t=torch.float32),
             workspace=z(4096, t=torch.uint8))
    a["workspace"] = a["workspace"][-a["workspace"].data_ptr() % 256:][:256]
    return {**a, **kw}


def test_its_arguments_reach_the_library(monkeypatch):
    # on the CPU (device -1) as far as the library's own checks: of a workspace that is too small, which comes last
    import torch
    got = []
    monkeypatch.setattr(_serving, "_call", lambda what, fn, index, stream, args: got.append(fn(*args, None)))
    _serving._attention(-1, None, *_args(max_seq_len=100000, window=50000).values())
    assert got.pop() == -3
    _serving._attention(-1, None, *_args(q=torch.zeros((0, 4, 64), dtype=torch.bfloat16), lse=None, idx_map=torch.zeros(
        2, dtype=torch.int32), out=torch.zeros((0, 4, 64), dtype=torch.bfloat16)).values())
    assert got.pop() == 0  # nothing to do
    _serving._attention(-1, None, *_args(max_seq_len=100000, window=0, sinks=0).values())
    assert got.pop() == -3
    for bad, rc in ((dict(window=-1), -1), (dict(sinks=-1), -1), (dict(max_seq_len=-1), -1), (dict(scale=-1.0), -1),
                    (dict(sinks=0, max_q_len=1 << 32), -1),
                    (dict(k_scale=torch.ones(2)), -1)):
        _serving._attention(-1, None, *_args(**bad).values())
        assert got.pop() == rc, bad


@pytest.mark.parametrize("bad", [dict(max_q_len=1 << 32), dict(max_seq_len=1 << 70), dict(window=2.5), dict(sinks=1 << 31),
                                 dict(sinks=0, window=2.5),
                                 dict(scale="x"), "q", "out", "block_table", "query_start", "seq_lens", "workspace", "lse",
                                 "k_pages", "v_pages"])
def test_its_refusals(monkeypatch, bad):
    monkeypatch.setattr(_serving, "_call", lambda *a: pytest.fail("called"))
    if isinstance(bad, str):  # that tensor in another type
        bad = {bad: _args()[bad].double()}
    with pytest.raises(mds.MdsError):
        _serving._attention(-1, None, *_args(**bad).values())
