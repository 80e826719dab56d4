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
    assert f(65535, 64, (1 << 24) - 1, 128, out) == 0 and tuple(out) == (0, 7, 5)  # (work-groups counted in 64 bits)


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


def _attention_plan(T, B, Hq, Hk, D, max_q, max_seq, window, sinks, dtype):
    """(rows, key groups, keys split)"""
    out = (ctypes.c_int32 * 4)()
    assert mds._lib().mds_debug_paged_attention_plan(T, B, Hq, Hk, D, max_q, max_seq, window, sinks, dtype, out) == 0
    assert out[2] >= 1 and out[3] >= 128 and out[3] % 128 == 0
    return out[0], out[1], out[2] > 1


def test_every_attention_variant_with_first_tokens_has_a_case():
    cases = set()
    for (rows, kg, kg8, split), ctx, chunk, Hq, Hk, _, window, sinks, _ in lc.ATTENTION_SINKS:
        for D in (64, 128):
            for dtype, groups in ((mds.BF16, kg), (mds.E4M3, kg8)):
                got = _attention_plan(sum(chunk), len(ctx), Hq, Hk, D, max(chunk), max(c + n for c, n in zip(ctx, chunk)),
                                      window, sinks, dtype)
                assert got == (rows, groups, split), (ctx[:3], D, dtype)
                cases.add((D, dtype, rows, groups))
    assert {r[0] for r, *_ in lc.ATTENTION_SINKS if r[3]} == {16, 32, 64, 128}  # joins
    reached = set()
    for B in (1, 3, 33, 40, 65, 128, 1000):
        for max_q in (1, 4, 8, 20, 100, 600, 2048):
            for Hk in (1, 2, 8):
                for G in (1, 3, 8):
                    for window, sinks in ((17, 1), (300, 64), (1000, 4), (2000, 16), (4096, 4), (20000, 10)):
                        for max_seq in (64, 300, 1300, 5000, 30000):
                            for D in (64, 128):
                                for dtype in (mds.BF16, mds.E4M3):
                                    if B * max_q <= 1 << 17:
                                        p = _attention_plan(B * max_q, B, G * Hk, Hk, D, max_q, max_seq, window, sinks, dtype)
                                        reached.add((D, dtype, *p[:2]))
    assert reached == cases and len(cases) == 36


def test_attention_plan_refusals():
    f, out = mds._lib().mds_debug_paged_attention_plan, (ctypes.c_int32 * 4)()
    ok = [8, 2, 4, 2, 64, 4, 100, 10, 2, mds.BF16, out]
    assert f(*ok) == 0
    for i, bad, rc in ((0, 0, -1), (0, -1, -1), (1, 0, -1), (2, 3, -1), (4, 80, -2), (5, 0, -1), (6, -1, -1), (7, -1, -1),
                       (8, -1, -1), (9, 0, -1), (10, None, -1)):
        assert f(*ok[:i], bad, *ok[i + 1:]) == rc, i
