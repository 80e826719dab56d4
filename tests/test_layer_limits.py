"""Calls past what a launch can hold (its threads are counted in 32 bits) are
refused on the host (no GPU)."""
import markov_draft_sampling_amd as mds

FAKE = 1 << 24  # never dereferenced: validation fails first


def _rope(T, Hq, Hk, D, append):
    q = [FAKE, (Hq + 2 * Hk) * D, D]
    args = [T, Hq, Hk, D, 16, *q, *q, *(q if append else []), FAKE, FAKE, None, None, 1e-6, 1.0, 0, FAKE, Hq * D, D]
    if append:
        pages = [16 * Hk * D, Hk * D, D]
        return mds._lib().mds_qk_norm_rope_append(*args, FAKE, FAKE, mds.BF16, 16, 8, *pages, *pages, FAKE, None, None, None, None)
    return mds._lib().mds_qk_norm_rope(*args, FAKE, Hk * D, D, None)


def test_rotations_of_too_many_heads():
    for T, Hq, Hk, D in ((1 << 24, 120, 7, 16), (1 << 24, 60, 60, 128), (1 << 21, 500, 100, 256)):
        assert _rope(T, Hq, Hk, D, False) == -2, (T, Hq, Hk, D)
        assert b"too many heads" in mds._lib().mds_last_error()
        assert _rope(T, max(Hq - Hk, 1), Hk, D, True) == -2, (T, Hq, Hk, D)
        assert b"too many heads" in mds._lib().mds_last_error()


def test_matrices_of_too_many_tiles():
    lib = mds._lib()
    for V, H in ((1 << 22, 32768), ((1 << 24) - 1, 65536), ((1 << 24) - 1, 8192)):
        n, m = mds.lm_head_mxfp4_bytes(V, H)
        codes, scales, tiled, ts = FAKE, FAKE + (1 << 40), FAKE + (1 << 41), FAKE + (1 << 42)
        assert lib.mds_tile_lm_head_mxfp4(V, H, codes, scales, tiled, n, ts, m, None) == -2
        assert b"too large" in lib.mds_last_error()
        assert lib.mds_quantize_lm_head_mxfp4(V, H, codes, tiled, n, ts, m, None) == -2
        assert b"too large" in lib.mds_last_error()
        assert lib.mds_unpack_lm_head_mxfp4(V, H, tiled, ts, codes, None) == -2
        assert b"too large" in lib.mds_last_error()


def test_logits_of_too_many_work_groups():
    lib = mds._lib()
    B, K, V, H = 65535, 64, 262000, 128
    assert lib.mds_lm_head_mxfp4(B, K, V, H, FAKE, H, FAKE, FAKE, FAKE, mds.BF16, K * V, V, None) == -2
    assert b"too many work-groups" in lib.mds_last_error()


def test_attention_of_too_many_work_groups():
    # (work-groups of four waves: four key groups, or the four row groups of a prompt's tile)
    lib = mds._lib()
    for T, B, Hq, Hk, max_q in ((65535, 65535, 1024, 1024, 1), (65535, 65535, 257, 257, 1), (1 << 22, 4, 1024, 1024, 1 << 20)):
        q, pages = [FAKE, Hq * 64, 64], [16 * Hk * 64, Hk * 64, 64]
        for window, sinks in ((0, 0), (4096, 4)):
            rc = lib.mds_paged_attention_sinks(T, B, Hq, Hk, 64, *q, FAKE, FAKE, mds.BF16, 16, 8, *pages, *pages, FAKE, B, 4096,
                                               None, FAKE, FAKE, max_q, 20000, 0.125, 1, window, sinks, None, None, *q, None, FAKE,
                                               1 << 50, None)
            assert rc == -2, (T, Hk, window)
            assert b"too many work-groups" in lib.mds_last_error()


def test_by_parts_frequencies_whose_pairs_are_all_slow_or_all_fast():
    # pairs that turn less than beta_slow times within the trained positions are divided by factor, the first one too; those
    # of more than beta_fast are kept
    import math
    import numpy as np
    for dim, base, trained, fast, slow in ((64, 10000.0, 6, 32.0, 1.0), (64, 10000.0, 1, 2.0, 0.5), (128, 5e5, 128, 64.0, 32.0),
                                           (16, 1.5, 1 << 20, 32.0, 1.0), (2, 10000.0, 3, 32.0, 1.0)):
        f, _ = mds.rope_frequencies(dim, base=base, device="cpu")
        g, _ = mds.rope_frequencies(dim, base=base, scaling="yarn", factor=8.0, trained_len=trained, beta_fast=fast,
                                    beta_slow=slow, device="cpu")
        turns, ratio = trained * f.numpy() / (2 * math.pi), g.numpy() / f.numpy()
        assert (turns < slow).all() or (turns > fast).all()
        assert np.allclose(ratio, 0.125 if turns[0] < slow else 1.0, rtol=1e-12), (dim, trained)
