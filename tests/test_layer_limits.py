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
