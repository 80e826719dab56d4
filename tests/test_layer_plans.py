"""Which variant of a kernel a call takes (host only, no GPU): every one that
some call takes is run by the cases of layer_cases.py."""
import ctypes

import pytest

import layer_cases as lc
import markov_draft_sampling_amd as mds


def _lm_head_plan(rows, V):
    out = (ctypes.c_int32 * 3)()
    assert mds._lib().mds_debug_lm_head_mxfp4_plan(rows, 1, V, 128, out) == 0
    return tuple(out)


def test_every_lm_head_variant_has_a_case():
    vocab = [2, 100, 515, *range(1000, 60000, 1777), *range(60000, 300000, 9001), *(1 << n for n in range(10, 24)),
             *(1000003 * n for n in range(1, 16, 3)), 100003, 128256, 151936, 200064]
    reached = {_lm_head_plan(rows, V) for V in vocab for rows in [*range(1, 300), 400, 577, 1000, 10000, 65535]}
    cases = {_lm_head_plan(rows, V) for V, some in lc.MXFP4_HEAD for rows in some}
    assert reached - cases == set()
    assert len(cases) == sum(len(some) for _, some in lc.MXFP4_HEAD) == 54  # and no two take the same


def test_lm_head_plan_refusals():
    f, out = mds._lib().mds_debug_lm_head_mxfp4_plan, (ctypes.c_int32 * 3)()
    assert f(1, 1, 1000, 128, None) == -1 and f(0, 1, 1000, 128, out) == -1 and f(1, 1, 1, 128, out) == -1
    assert f(1, 1, 1000, 200, out) == -2
    with pytest.raises(ctypes.ArgumentError):
        f(1, 1, 1000, "128", out)


def test_every_rotation_variant_has_a_case():
    def plan(T, Hq, Hk, D, append):
        out = (ctypes.c_int32 * 2)()
        assert mds._lib().mds_debug_qk_norm_rope_plan(T, Hq, Hk, D, append, out) == 0
        return tuple(out)
    cases = set()
    for T, Hq, Hk, D, _, _, _, to, short in lc.ROPE:
        long, brief = (plan(n, Hq, Hk, D, to != "rows") for n in (T, short))
        assert long[0] == brief[0] and (long[1], brief[1]) == (2, 1)
        cases |= {(*long, to), (*brief, to)}
    assert len(cases) == 18
    reached = {(*plan(T, Hq, Hk, D, to != "rows"), to) for T in (0, 1, 300, 5000, 1 << 20) for Hq in (1, 8, 100)
               for Hk in (1, 8) for D in range(16, 257, 16) for to in ("rows", "bf16", "e4m3")}
    assert reached == cases


def test_rotation_plan_refusals():
    f, out = mds._lib().mds_debug_qk_norm_rope_plan, (ctypes.c_int32 * 2)()
    assert f(1, 1, 1, 64, 0, None) == -1 and f(-1, 1, 1, 64, 0, out) == -1 and f(1, 0, 1, 64, 0, out) == -1
    assert f(1, 1, 1, 72, 0, out) == -2 and f(1 << 24, 100, 50, 64, 1, out) == -2
