"""Host-side checks of the serving operators (no GPU): sizes, strides, dtypes
and pointers are refused before any device work, and the workspace queries."""
import pytest

import markov_draft_sampling_amd as mds

FAKE = 1 << 24  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    return mds._lib()


def _tables(**kw):
    a = dict(B=4, n_slots=8, max_pages=16, page_size=16, n_pages=64, max_tokens=64, idx_map=FAKE, kv_len=FAKE,
             advance=None, advance_add=0, chunk_len=FAKE, block_table=FAKE, pages_held=FAKE, free_list=FAKE,
             free_count=FAKE, query_start=FAKE, seq_lens=FAKE, positions=FAKE, slot_map=FAKE, kv_len_out=FAKE,
             pages_held_out=FAKE, free_count_out=FAKE, status=None, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,rc", [(dict(B=0), -1), (dict(B=65536), -1), (dict(n_slots=0), -1),
                                   (dict(n_slots=(1 << 17) + 1), -1), (dict(idx_map=None, n_slots=3), -1),
                                   (dict(page_size=0), -1), (dict(page_size=24), -2), (dict(page_size=8), -2),
                                   (dict(page_size=2048), -2), (dict(max_pages=0), -1), (dict(max_pages=1 << 27), -1),
                                   (dict(n_pages=0), -1), (dict(max_tokens=-1), -1), (dict(kv_len=None), -1),
                                   (dict(block_table=None), -1), (dict(slot_map=None), -1),
                                   (dict(free_count_out=None), -1)])
def test_page_tables_refusals(lib, kw, rc):
    assert lib.mds_kv_page_tables(*_tables(**kw)) == rc
    assert lib.mds_last_error()


def _append(**kw):
    a = dict(T=4, Hkv=2, D=64, k=FAKE, kts=128, khs=64, v=FAKE, vts=128, vhs=64, kp=FAKE, vp=FAKE, dt=1, page=16,
             n_pages=8, kps=2048, kss=128, kph=64, vps=2048, vss=128, vph=64, slot=FAKE, ksc=None, vsc=None, st=None,
             stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,rc", [(dict(T=-1), -1), (dict(Hkv=0), -1), (dict(D=40), -2), (dict(D=0), -1),
                                   (dict(dt=0), -1), (dict(dt=2), -1), (dict(dt=3), -1), (dict(k=None), -1),
                                   (dict(slot=None), -1), (dict(page=20), -2), (dict(k=FAKE + 2), -2),
                                   (dict(kts=129), -2), (dict(vhs=-64), -1), (dict(kp=FAKE + 8), -2),
                                   (dict(kss=100), -2), (dict(kss=64, kph=64), -1), (dict(vps=128), -1),
                                   (dict(kps=-2048), -1),
                                   (dict(T=1 << 24, Hkv=1024, kps=1 << 20, kss=1 << 16, vps=1 << 20, vss=1 << 16),
                                    -2)])
def test_append_refusals(lib, kw, rc):
    assert lib.mds_kv_append(*_append(**kw)) == rc


def test_append_of_nothing_is_ok(lib):
    assert lib.mds_kv_append(*_append(T=0, k=None, v=None, slot=None)) == 0


def _attend(**kw):
    a = dict(T=8, B=2, Hq=4, Hkv=2, D=64, q=FAKE, qts=256, qhs=64, kp=FAKE, vp=FAKE, dt=1, page=16, n_pages=8, kps=2048,
             kss=128, kph=64, vps=2048, vss=128, vph=64, table=FAKE, n_slots=2, max_pages=4, idx=None, qs=FAKE, seq=FAKE,
             mq=4, ms=64, scale=0.125, causal=1, window=0, ksc=None, vsc=None, out=FAKE, ots=256, ohs=64, lse=None,
             ws=FAKE, wsb=1 << 30, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,rc", [(dict(T=-1), -1), (dict(B=0), -1), (dict(Hq=5), -1), (dict(Hkv=0), -1),
                                   (dict(D=80), -2), (dict(D=256), -2), (dict(D=0), -1), (dict(q=None), -1),
                                   (dict(ws=None), -1), (dict(table=None), -1), (dict(dt=0), -1), (dict(page=8), -2),
                                   (dict(n_slots=1), -1), (dict(mq=-1), -1), (dict(ms=-1), -1), (dict(ms=1 << 31), -1),
                                   (dict(window=-1), -1), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1),
                                   (dict(scale=float("inf")), -1), (dict(causal=2), -1), (dict(ksc=FAKE), -1),
                                   (dict(q=FAKE + 4), -2), (dict(ots=100), -2), (dict(ots=64, ohs=64), -1),
                                   (dict(ohs=-64), -1), (dict(ws=FAKE + 16), -1), (dict(wsb=16), -3),
                                   (dict(kps=2047), -2), (dict(vss=-128), -1)])
def test_attention_refusals(lib, kw, rc):
    assert lib.mds_paged_attention(*_attend(**kw)) == rc


def test_attention_of_nothing_is_ok(lib):
    assert lib.mds_paged_attention(*_attend(T=0, q=None, out=None)) == 0


def test_the_stride_of_a_dimension_of_one_is_not_looked_at(lib):
    # calls that end before any device work: nothing to do, or (the last check) a workspace that is too small
    one = dict(n_pages=1, kps=7, vps=-3)
    assert lib.mds_kv_append(*_append(T=0, Hkv=1, k=None, v=None, slot=None, kts=3, vts=-1, khs=-5, vhs=9, kph=-2, vph=5,
                                      **one)) == 0
    heads = dict(Hq=1, Hkv=1, qhs=3, ohs=-7, kph=1, vph=-9)
    assert lib.mds_paged_attention(*_attend(T=1, mq=0, qts=5, ots=-1, **heads, **one)) == 0
    assert lib.mds_paged_attention(*_attend(T=2, mq=0, qts=5, **heads, **one)) == -2
    assert lib.mds_lm_head_fp8(*_head(B=1, K=1, hrs=3, rs=-1, ss=7, wsb=16)) == -3
    assert lib.mds_lm_head_fp8(*_head(B=1, K=2, hrs=3, rs=-1, wsb=16)) == -1


def test_attention_workspace_bytes():
    n = mds.paged_attention_workspace_bytes
    assert n(1, 1, 8, 8, 128, 1, 1) >= 256
    # long keys of few rows are split; the partials of a split are float32 rows of D + 2
    assert n(1, 1, 32, 8, 128, 1, 131072) > n(1, 1, 32, 8, 128, 1, 128)
    with pytest.raises(mds.MdsError, match="unsupported"):
        n(1, 1, 8, 8, 96, 1, 64)
    with pytest.raises(mds.MdsError, match="invalid argument"):
        n(1, 1, 8, 3, 128, 1, 64)


def test_attention_workspace_of_the_largest_step_serves_smaller_ones():
    import random
    rng = random.Random(0)
    n = mds.paged_attention_workspace_bytes
    log = lambda hi: int(round(hi ** rng.random()))  # noqa: E731
    # fewer tokens, whose keys are split, beside a prompt, whose keys are not
    assert n(2048, 8, 32, 8, 128, 2048, 16384) >= n(8, 8, 32, 8, 128, 1, 16384) > 256
    for _ in range(20000):
        hk, g, D = log(64), rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([64, 128])
        T, B, q, s = log(20000), log(500), log(4000), log(1 << 20)
        window = rng.choice([0, 0, log(20000)])
        t, b, r, u = rng.randint(0, T), rng.randint(1, B), rng.randint(0, q), rng.randint(0, s)
        assert n(t, b, hk * g, hk, D, r, u, window) <= n(T, B, hk * g, hk, D, q, s, window)


def _head(**kw):
    a = dict(B=2, K=3, V=1000, H=256, hidden=FAKE, hrs=256, lm=FAKE, sc=FAKE, out=FAKE, dt=0, rs=3000, ss=1000, ws=FAKE,
             wsb=1 << 30, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,rc", [(dict(B=0), -1), (dict(K=0), -1), (dict(K=65), -1), (dict(V=1), -1),
                                   (dict(H=200), -2), (dict(H=64), -1), (dict(hidden=None), -1), (dict(sc=None), -1),
                                   (dict(dt=2), -1), (dict(hrs=248), -1), (dict(hrs=260), -1), (dict(lm=FAKE + 8), -1),
                                   (dict(ss=999), -1), (dict(rs=2000), -1), (dict(ws=FAKE + 8), -1), (dict(wsb=16), -3)])
def test_lm_head_fp8_refusals(lib, kw, rc):
    assert lib.mds_lm_head_fp8(*_head(**kw)) == rc


def test_fp8_matrix_sizes_and_refusals(lib):
    assert mds.lm_head_fp8_tiled_bytes(200064, 4096) == 200064 * 4096
    assert mds.lm_head_fp8_tiled_bytes(17, 128) == 32 * 128
    with pytest.raises(mds.MdsError, match="unsupported"):
        mds.lm_head_fp8_tiled_bytes(1000, 130)
    need = 1008 * 256
    assert lib.mds_tile_lm_head_fp8(1000, 256, None, FAKE, need, None) == -1
    assert lib.mds_tile_lm_head_fp8(1000, 256, FAKE, FAKE + (1 << 20), need - 1, None) == -1
    assert lib.mds_tile_lm_head_fp8(1000, 256, FAKE, FAKE + 1024, need, None) == -1  # overlap
    assert lib.mds_tile_lm_head_fp8(1000, 256, FAKE + 4, FAKE + (1 << 20), need, None) == -1
    assert lib.mds_quantize_lm_head_fp8(1000, 256, FAKE, FAKE + (1 << 20), need, None, None) == -1
    assert lib.mds_quantize_lm_head_fp8(1000, 256, FAKE, FAKE + (1 << 18), need, FAKE, None) == -1  # overlap


def test_unknown_attribute_still_raises():
    with pytest.raises(AttributeError):
        mds.no_such_operator
    assert callable(mds.paged_attention)


def _pack(args):
    import struct
    return b"".join(struct.pack("d" if isinstance(x, float) else "q", 0 if x is None else x) for x in args)


@pytest.mark.parametrize("name,make,bad", [("mds_kv_page_tables", _tables, dict(page_size=24)),
                                           ("mds_kv_append", _append, dict(D=20)),
                                           ("mds_paged_attention", _attend, dict(D=96)),
                                           ("mds_lm_head_fp8", _head, dict(H=100))])
def test_packed_calls_refuse_as_the_calls_do(lib, name, make, bad):
    call = ["mds_kv_page_tables", "mds_kv_append", "mds_paged_attention", "mds_lm_head_fp8"].index(name)
    args = make(**bad)
    rc = getattr(lib, name)(*args)
    message = lib.mds_last_error()
    n = len(args) - 1
    assert rc < 0 and lib.mds_call_packed(call, _pack(args[:-1]), n, None) == rc
    assert lib.mds_last_error() == message
    assert lib.mds_call_packed(call, _pack(args[:-1]), n - 1, None) == -1
    assert lib.mds_call_packed(call, _pack(args), n + 1, None) == -1
    assert lib.mds_call_packed(call, _pack([1 << 40] + args[1:-1]), n, None) == -1
    assert lib.mds_call_packed(9, _pack(args[:-1]), n, None) == -1
    assert lib.mds_call_packed(call, None, n, None) == -1
    assert b"NULL" in lib.mds_last_error()


def test_the_three_copies_of_a_signature_agree():
    # the header's prototype, the binding's ctypes signature and the packed call's type string
    import ctypes
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(mds.__file__)))
    with open(os.path.join(root, "include", "mds.h")) as f:
        header = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    with open(os.path.join(root, "markov_draft_sampling_amd", "csrc", "abi_serve.hip")) as f:
        strings = re.findall(r'"([iplzf]{10,})"', f.read())
    ctype = {"i": ctypes.c_int, "l": ctypes.c_int64, "p": ctypes.c_void_p, "z": ctypes.c_size_t, "f": ctypes.c_float}
    calls = ["mds_kv_page_tables", "mds_kv_append", "mds_paged_attention", "mds_lm_head_fp8"]
    assert len(strings) == len(calls)
    for name, packed in zip(calls, strings):
        args = re.search(name + r"\((.*?)\);", header, re.S).group(1).split(",")
        kinds = ["p" if "*" in a else {"int": "i", "int64_t": "l", "size_t": "z", "float": "f"}[a.split()[0]] for a in args]
        assert "".join(kinds) == packed + "p", name  # the stream is not packed
        types = mds._SIGS[name][0]
        assert len(types) == len(kinds), name
        for kind, t in zip(kinds, types):
            assert t is ctype[kind] or ctypes.sizeof(t) == ctypes.sizeof(ctype[kind]) and t._type_ == ctype[kind]._type_, name
