"""Host-side checks of the operators of a layer's step (no GPU): what is
refused before any device work, sizes, frequencies, and the copies of each
signature against each other."""
import ctypes
import math
import os
import re
import sys

import numpy as np
import pytest

import layer_ref as lr
import markov_draft_sampling_amd as mds

FAKE = 1 << 24  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    return mds._lib()


def _rope(**kw):
    a = dict(T=4, Hq=4, Hk=2, D=64, R=64, q=FAKE, qts=512, qhs=64, k=FAKE, kts=512, khs=64, pos=FAKE, freq=FAKE, qw=FAKE,
             kw=FAKE, eps=1e-6, rs=1.0, il=0, qo=FAKE, qots=256, qohs=64, ko=FAKE, kots=128, kohs=64, stream=None)
    a.update(kw)
    return list(a.values())


_ROPE_BAD = [(dict(T=-1), -1), (dict(T=(1 << 24) + 1), -1), (dict(Hq=0), -1), (dict(Hq=1025), -1), (dict(Hk=0), -1),
             (dict(D=0), -1), (dict(D=40), -2), (dict(D=272), -2), (dict(R=-16), -1), (dict(R=80), -1), (dict(R=24), -2),
             (dict(q=None), -1), (dict(k=None), -1), (dict(pos=None), -1), (dict(freq=None), -1), (dict(qo=None), -1),
             (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
             (dict(rs=float("nan")), -1), (dict(rs=float("inf")), -1), (dict(il=2), -1), (dict(qw=FAKE + 8), -1),
             (dict(kw=FAKE + 2), -1), (dict(pos=FAKE + 4), -1), (dict(freq=FAKE + 4), -1), (dict(q=FAKE + 8), -2),
             (dict(qts=100), -2), (dict(khs=-64), -1), (dict(qo=FAKE + 8), -2), (dict(qots=128), -1), (dict(qohs=32), -1),
             (dict(T=1 << 24, Hq=200), -2)]


@pytest.mark.parametrize("kw,rc", _ROPE_BAD + [(dict(ko=None), -1), (dict(kots=64), -1), (dict(ko=FAKE + 4), -2)])
def test_rope_refusals(lib, kw, rc):
    assert lib.mds_qk_norm_rope(*_rope(**kw)) == rc
    assert lib.mds_last_error()


def _rope_append(**kw):
    a = dict(T=4, Hq=4, Hk=2, D=64, R=64, q=FAKE, qts=512, qhs=64, k=FAKE, kts=512, khs=64, v=FAKE, vts=512, vhs=64,
             pos=FAKE, freq=FAKE, qw=FAKE, kw=FAKE, eps=1e-6, rs=1.0, il=0, qo=FAKE, qots=256, qohs=64, kp=FAKE, vp=FAKE,
             dt=1, page=16, n_pages=8, kps=2048, kss=128, kph=64, vps=2048, vss=128, vph=64, slot=FAKE, ksc=None, vsc=None,
             st=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,rc", _ROPE_BAD + [(dict(v=None), -1), (dict(slot=None), -1), (dict(kp=None), -1),
                                               (dict(vp=None), -1), (dict(dt=0), -1), (dict(dt=2), -1), (dict(page=8), -2),
                                               (dict(n_pages=0), -1), (dict(vts=-8), -1), (dict(vhs=4), -2),
                                               (dict(kp=FAKE + 8), -2), (dict(kss=100), -2), (dict(kss=64, kph=64), -1),
                                               (dict(vps=128), -1)])
def test_rope_append_refusals(lib, kw, rc):
    assert lib.mds_qk_norm_rope_append(*_rope_append(**kw)) == rc
    assert lib.mds_last_error()


def test_rope_of_nothing_is_ok(lib):
    none = dict(T=0, q=None, k=None, pos=None, qo=None)
    assert lib.mds_qk_norm_rope(*_rope(ko=None, **none)) == 0
    assert lib.mds_qk_norm_rope_append(*_rope_append(v=None, slot=None, **none)) == 0
    # the stride of a dimension of one is not looked at; no frequencies are needed where nothing turns
    assert lib.mds_qk_norm_rope(*_rope(Hk=1, R=0, freq=None, khs=-3, kohs=5, kots=7, qts=9, ko=None, **none)) == 0


def _attend(**kw):
    a = dict(T=8, B=2, Hq=4, Hkv=2, D=64, q=FAKE, qts=256, qhs=64, kp=FAKE, vp=FAKE, dt=1, page=16, n_pages=8, kps=2048,
             kss=128, kph=64, vps=2048, vss=128, vph=64, table=FAKE, n_slots=2, max_pages=4, idx=None, qs=FAKE, seq=FAKE,
             mq=4, ms=64, scale=0.125, causal=1, window=16, sinks=4, ksc=None, vsc=None, out=FAKE, ots=256, ohs=64,
             lse=None, ws=FAKE, wsb=1 << 30, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,rc", [(dict(sinks=-1), -1), (dict(sinks=(1 << 29) + 1), -1), (dict(window=-1), -1),
                                   (dict(D=80), -2), (dict(q=None), -1), (dict(wsb=16), -3), (dict(causal=2), -1),
                                   (dict(out=FAKE + 4), -2)])
def test_attention_sinks_refusals(lib, kw, rc):
    assert lib.mds_paged_attention_sinks(*_attend(**kw)) == rc
    assert lib.mds_last_error()


def test_attention_sinks_workspace_bytes():
    n = mds.paged_attention_workspace_bytes
    assert n(8, 1, 32, 8, 128, 8, 1 << 20, 1000, 0) == n(8, 1, 32, 8, 128, 8, 1 << 20, 1000)
    assert n(8, 1, 32, 8, 128, 8, 1 << 20, 0, 64) == n(8, 1, 32, 8, 128, 8, 1 << 20)  # no window: all is seen
    assert n(8, 1, 32, 8, 128, 8, 1 << 20, 1000, 5000) >= n(8, 1, 32, 8, 128, 8, 1 << 20, 1000, 4)
    assert n(8, 1, 32, 8, 128, 8, 1 << 30, 1 << 30, 1 << 29) > 0
    with pytest.raises(mds.MdsError, match="sinks"):
        n(8, 1, 32, 8, 128, 8, 100, 10, -1)


def _head(**kw):
    a = dict(B=2, K=3, V=1000, H=256, hidden=FAKE, hrs=256, lm=FAKE, sc=FAKE, out=FAKE, dt=0, rs=3000, ss=1000, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,rc", [(dict(B=0), -1), (dict(K=0), -1), (dict(K=65), -1), (dict(V=1), -1),
                                   (dict(H=200), -2), (dict(H=64), -1), (dict(hidden=None), -1), (dict(sc=None), -1),
                                   (dict(lm=None), -1), (dict(out=None), -1), (dict(dt=2), -1), (dict(hrs=248), -1),
                                   (dict(hrs=260), -1), (dict(hrs=(1 << 22) + 8), -2), (dict(lm=FAKE + 8), -1),
                                   (dict(sc=FAKE + 2), -1), (dict(hidden=FAKE + 8), -1), (dict(ss=999), -1),
                                   (dict(rs=2000), -1),
                                   (dict(B=65535, K=64, V=(1 << 24) - 1, rs=1 << 30, ss=1 << 24), -2)])
def test_lm_head_mxfp4_refusals(lib, kw, rc):
    assert lib.mds_lm_head_mxfp4(*_head(**kw)) == rc
    assert lib.mds_last_error()


def test_mxfp4_matrix_sizes_and_refusals(lib):
    assert mds.lm_head_mxfp4_bytes(200064, 4096) == (200064 * 2048, 200064 * 128)
    assert mds.lm_head_mxfp4_bytes(17, 128) == (32 * 64, 2 * 256)
    with pytest.raises(mds.MdsError, match="unsupported"):
        mds.lm_head_mxfp4_bytes(1000, 130)
    n, m = mds.lm_head_mxfp4_bytes(1000, 256)
    t, s = FAKE + (1 << 22), FAKE + (1 << 23)
    tile, quant, unpack = lib.mds_tile_lm_head_mxfp4, lib.mds_quantize_lm_head_mxfp4, lib.mds_unpack_lm_head_mxfp4
    sc = FAKE + (1 << 21)
    assert tile(1000, 256, None, sc, t, n, s, m, None) == -1
    assert tile(1000, 256, FAKE, None, t, n, s, m, None) == -1
    assert tile(1000, 256, FAKE, sc, t, n - 1, s, m, None) == -1
    assert tile(1000, 256, FAKE, sc, t, n, s, m - 1, None) == -1
    assert tile(1000, 256, FAKE + 4, sc, t, n, s, m, None) == -1
    assert tile(1000, 256, FAKE, sc, t + 8, n, s, m, None) == -1
    assert tile(1000, 256, FAKE, sc, t, n, s + 2, m, None) == -1
    assert tile(1000, 256, FAKE, sc, t, n, t + n - 16, m, None) == -1  # overlaps
    assert tile(1000, 256, t, sc, t, n, s, m, None) == -1
    assert tile(1000, 256, FAKE, t + 64, t, n, s, m, None) == -1
    assert quant(1000, 256, None, t, n, s, m, None) == -1
    assert quant(1000, 256, FAKE + 2, t, n, s, m, None) == -1
    assert quant(1000, 256, t - 16, t, n, s, m, None) == -1
    assert unpack(1000, 256, t, s, None, None) == -1
    assert unpack(1000, 256, None, s, FAKE, None) == -1
    assert unpack(1000, 256, t, s, s + 16, None) == -1


_CALLS = [("mds_paged_attention_sinks", _attend), ("mds_qk_norm_rope", _rope), ("mds_qk_norm_rope_append", _rope_append),
          ("mds_lm_head_mxfp4", _head)]


def test_the_copies_of_a_signature_agree():
    # the header's prototype and the binding's ctypes signature
    root = os.path.dirname(os.path.dirname(os.path.abspath(mds.__file__)))
    with open(os.path.join(root, "include", "mds.h")) as f:
        header = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    ctype = {"i": ctypes.c_int, "l": ctypes.c_int64, "p": ctypes.c_void_p, "z": ctypes.c_size_t, "f": ctypes.c_float, "d": ctypes.c_double}
    for name, make in _CALLS:
        args = re.search(name + r"\((.*?)\);", header, re.S).group(1).split(",")
        kinds = ["p" if "*" in a else {"int": "i", "int64_t": "l", "size_t": "z", "float": "f", "double": "d"}[a.split()[0]] for a in args]
        assert [t._type_ for t in mds._SIGS[name][0]] == [ctype[k]._type_ for k in kinds], name
        assert len(make()) == len(kinds)


def test_the_compiled_calls_check_their_arguments():
    import torch
    from markov_draft_sampling_amd import _serving
    calls = _serving._calls()
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    for fn, n in ((calls.qk_norm_rope, 12), (calls.qk_norm_rope_append, 18), (calls.paged_attention, 19),
                  (calls.lm_head_mxfp4, 6)):
        with pytest.raises(mds.MdsError, match="number of arguments"):
            fn(*[x] * (n - 1))
        with pytest.raises(mds.MdsError, match="number of arguments"):
            fn()
        with pytest.raises(mds.MdsError, match="GPU"):
            fn(*[x] * n)
        for bad in (None, 3, "q", [x]):
            with pytest.raises(mds.MdsError, match="must be a tensor"):
                fn(*[bad] * n)
    held = sys.getrefcount(x)
    for _ in range(100):
        with pytest.raises(mds.MdsError):
            calls.lm_head_mxfp4(x, x, x, x, None, None)
    assert sys.getrefcount(x) == held


def test_frequencies():
    f, s = mds.rope_frequencies(64, device="cpu")
    assert s == 1.0 and f.dtype.itemsize == 8 and f.shape == (32,)
    assert np.allclose(f.numpy(), 10000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    g, s = mds.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert s == 1.0 and np.allclose(g.numpy(), f.numpy() / 4, rtol=1e-15)
    g, s = mds.rope_frequencies(64, scaling="ntk", factor=4.0, device="cpu")
    assert s == 1.0 and g[0] == f[0] and np.isclose(float(g[-1]), float(f[-1]) / 4, rtol=1e-12)
    g, s = mds.rope_frequencies(128, base=5e5, scaling="yarn", factor=8.0, trained_len=8192, device="cpu")
    f, _ = mds.rope_frequencies(128, base=5e5, device="cpu")
    assert np.isclose(s, 1 + 0.1 * math.log(8.0), rtol=1e-15)
    turns = 8192 * f.numpy() / (2 * math.pi)
    ratio = g.numpy() / f.numpy()
    assert np.allclose(ratio[turns > 40], 1.0, rtol=1e-12) and np.allclose(ratio[turns < 0.8], 0.125, rtol=1e-12)
    assert (np.diff(ratio) <= 1e-15).all() and ((ratio > 0.126) & (ratio < 0.999)).sum() > 5
    g, s = mds.rope_frequencies(128, base=5e5, scaling="yarn", factor=1.0, trained_len=8192, device="cpu")
    assert s == 1.0 and np.allclose(g.numpy(), f.numpy(), rtol=1e-15)
    for bad in (dict(rotary_dim=63), dict(rotary_dim=0), dict(factor=0.5), dict(scaling="other"), dict(base=1.0),
                dict(scaling="yarn"), dict(scaling="yarn", trained_len=10, beta_fast=1.0), dict(rotary_dim=2, scaling="ntk")):
        with pytest.raises(mds.MdsError):
            mds.rope_frequencies(**{"rotary_dim": 64, "device": "cpu", **bad})


def test_tensors_off_the_gpu_are_refused():
    import torch
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(mds.MdsError, match="GPU"):
        mds.qk_norm_rope(x, x, torch.zeros(2, dtype=torch.int64), None, x, x)
    with pytest.raises(mds.MdsError, match="GPU"):
        mds.lm_head_mxfp4(x[0], x, x, x, 1)
    with pytest.raises(mds.MdsError, match="GPU"):
        mds.quantize_lm_head_mxfp4(x[0])


def test_the_oracle_of_the_4_bit_format():
    # the reference itself, on values whose codes are known
    w = np.zeros((2, 64), np.float32)
    w[0, :8] = [7.9, 0.25, 0.75, 2.5, 3.5, 5.0, -5.01, -0.3]
    w[0, 32] = 2.0 ** -120
    w[1, :2] = [1.0, 0.125]
    codes, scales = lr.mx_quantize(w)
    assert codes[0, :8].tolist() == [7, 0, 2, 4, 6, 6, 15, 9] and scales[0].tolist() == [127, 25]
    assert codes[1, :2].tolist() == [6, 1] and scales[1, 0] == 125 and codes[0, 32] == 0
    v = lr.mx_values(codes, scales)
    assert v[0, :8].tolist() == [6, 0, 1, 2, 4, 4, -6, -0.5] and v[1, 1] == 0.125
    tiled, ts = lr.mx_tiles(codes.repeat(2, 1), scales.repeat(2, 1))
    assert tiled.shape == (1, 1024) and ts.shape == (1, 256)
    assert (lr.mx_pack(codes)[0, :2] == [7, 0x42]).all()
