"""Paged attention on the GPU against the float64 reference within bounds
derived from its roundings: head layouts, ragged and empty requests, masks
that leave a row nothing, windows, page sizes, strides, both cache types,
split and unsplit keys, stale memory behind the sequences."""
from __future__ import annotations

import math

import numpy as np
import pytest

import serving_ref as sr

pytestmark = pytest.mark.gpu


def _case(ctx, chunk, Hq, Hk, D, P, cache="bf16", causal=True, window=0, pad=3, seed=0, layout="nhd", idx=False,
          scale=None, poison=True, max_q=None, max_seq=None, qgain=1.5, q_layout="thd"):
    """Runs the call and the reference; returns (out, lse, reference tuple, tolerance inputs)."""
    import torch
    import markov_draft_sampling_amd as mds
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    B = len(ctx)
    seq = [a + n for a, n in zip(ctx, chunk)]
    held = [max(1, -(-x // P)) for x in seq]
    NP = sum(held) + 2
    pages = rng.permutation(NP - 1) + 1  # page 0 belongs to nobody
    MP = max(held) + 2
    n_slots = B + 4 if idx else B
    slots = rng.permutation(n_slots)[:B] if idx else np.arange(B)
    table = np.full((n_slots, MP), -123456, np.int32)  # garbage behind the pages
    at = 0
    for b in range(B):
        table[slots[b], :held[b]] = pages[at:at + held[b]]
        at += held[b]
    T = sum(chunk)
    q = (torch.randn((T + pad, Hq, D), generator=g) * qgain).to(torch.bfloat16)
    kv, dev = [], []
    for _ in range(2):
        x = torch.randn((NP, P, Hk, D), generator=g)
        if cache == "e4m3":
            x = (x * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
        else:
            x = x.to(torch.bfloat16)
        kv.append(x.float())
        d = x.clone()
        if poison:  # nothing behind a sequence's end may be read into a result
            nan = torch.tensor(float("nan")).to(x.dtype)
            for b in range(B):
                for p in range(seq[b], held[b] * P):
                    d.view(torch.uint8 if cache == "e4m3" else x.dtype)[table[slots[b], p // P], p % P] = \
                        nan.view(torch.uint8) if cache == "e4m3" else nan
            d.view(torch.uint8 if cache == "e4m3" else x.dtype)[0] = nan.view(torch.uint8) if cache == "e4m3" else nan
        d = d.cuda()
        if layout == "hnd":
            d = d.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(d.dtype) if cache == "e4m3" \
                else d.transpose(1, 2).contiguous().transpose(1, 2)
        elif layout == "padded":
            wide = torch.zeros((NP, P, Hk + 1, D + 32), dtype=torch.uint8 if cache == "e4m3" else d.dtype, device="cuda")
            wide[:, :, :Hk, :D] = d.view(wide.dtype)
            d = wide.view(d.dtype)[:, :, :Hk, :D]
        dev.append(d)
    ks = vs = None
    if cache == "e4m3":
        ks = torch.tensor(rng.uniform(0.9, 1.1, Hk) / 60, dtype=torch.float32)
        vs = torch.tensor(rng.uniform(0.9, 1.1, Hk) / 60, dtype=torch.float32)
    qs = np.concatenate([[0], np.cumsum(chunk)]).astype(np.int32)
    qd = q.cuda()
    out = torch.full((T + pad, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    if q_layout == "htd":
        qd = qd.transpose(0, 1).contiguous().transpose(0, 1)
        out = out.transpose(0, 1).contiguous().transpose(0, 1)
    lse = torch.full((T + pad, Hq), 7.0, device="cuda")
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    args = dict(scale=scale, causal=causal, window=window, idx_map=t(slots) if idx else None,
                k_scale=None if ks is None else ks.cuda(), v_scale=None if vs is None else vs.cuda(), lse=lse)
    mq = max(chunk) if max_q is None else max_q
    ms = max(seq) if max_seq is None else max_seq
    print(f"paged attention ctx {list(ctx)[:6]} chunk {list(chunk)[:6]} Hq {Hq} Hk {Hk} D {D} P {P} {cache} "
          f"causal {causal} window {window}", flush=True)
    ws = mds.paged_attention(qd, dev[0], dev[1], t(table), t(qs), t(seq), out, mq, ms, **args)
    torch.cuda.synchronize()
    assert mds.workspace_status(ws) == 0
    sc = 1 / math.sqrt(D) if scale is None else scale
    ref = sr.attention(q, kv[0], kv[1], table, qs, seq, sc, causal, window, slots if idx else None, ks, vs)
    again = out.clone()
    mds.paged_attention(qd, dev[0], dev[1], t(table), t(qs), t(seq), out, mq, ms, workspace=ws, **args)
    assert torch.equal(again, out)  # equal inputs, equal bits
    o, z = out.cpu(), lse.cpu()
    assert (o[T:] == 7.0).all() and (z[T:] == 7.0).all()  # rows behind the last token
    _check(o[:T], z[:T], ref, D, max(seq), T)
    return o, z


def _check(o, z, ref, D, L, T):
    import torch
    r, rl, A, S = (x[:T] for x in ref)
    tol, ltol = sr.attention_tolerance(r, A, S, D, L)
    err = (o.double() - r).abs()
    assert (err <= tol).all(), (float((err / tol).max()), torch.nonzero(err > tol)[:4].tolist())
    none = rl == -math.inf
    assert (z[none] == -math.inf).all() and (o[none] == 0).all()
    e = (z.double() - rl).abs()[~none]
    assert (e <= ltol[~none]).all(), float((e / ltol[~none]).max())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (8, 2), (6, 2), (5, 1), (16, 16)])
def test_single_tokens(D, cache, Hq, Hk):
    _case([0, 1, 15, 16, 31, 32, 33, 200, 511], [1] * 9, Hq, Hk, D, 16, cache)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("G", [1, 3, 4, 8])
def test_verification_chunks(D, cache, G):
    _case([0, 5, 30, 100, 333], [8, 8, 8, 8, 8], 2 * G, 2, D, 32, cache, seed=G)


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 7), (True, 40), (False, 20),
                                           (True, 10 ** 6)])
def test_masks(causal, window):
    _case([0, 3, 17, 64, 250], [7, 0, 5, 9, 1], 4, 2, 64, 16, causal=causal, window=window, seed=3)


@pytest.mark.parametrize("P", [16, 32, 128, 1024])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "padded"])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_pages_and_strides(P, layout, cache):
    _case([0, 100, 300], [3, 4, 2], 4, 2, 128, P, cache, layout=layout, idx=True, seed=P)


@pytest.mark.parametrize("D,cache", [(64, "bf16"), (128, "bf16"), (64, "e4m3"), (128, "e4m3")])
def test_prompt_chunks(D, cache):
    _case([0, 40, 130], [150, 1, 77], 4, 2, D, 16, cache, seed=9, q_layout="htd")


def test_prompt_with_window_and_both_ways():
    _case([100], [130], 3, 1, 64, 16, window=50, seed=1)
    _case([100], [130], 3, 1, 128, 16, causal=False, seed=2)


def test_split_keys_and_wrong_guess_of_the_longest():
    # the keys split over work-groups; a guess that is too small or too large changes nothing but rounding
    for ms in (None, 100, 40000):
        _case([2000, 900, 10], [2, 1, 3], 4, 1, 128, 16, seed=4, max_seq=ms)
    _case([3000], [1], 2, 2, 64, 64, "e4m3", seed=5)
    _case([5000], [2], 1, 1, 64, 16, window=700, seed=5)


def test_many_requests_and_empty_ones():
    rng = np.random.default_rng(0)
    ctx = rng.integers(0, 60, 130).tolist()
    chunk = rng.choice([0, 1, 2, 8], 130).tolist()
    _case(ctx, chunk, 2, 1, 64, 16, seed=6)
    chunk[77] = 90  # one prompt among them: tiles are found by row offset
    _case(ctx, chunk, 2, 1, 64, 16, seed=7)


@pytest.mark.parametrize("B", [65, 300, 4500])
def test_prompts_among_many_requests(B):
    # tiles found by row offset in one, two and three rounds of 64 probes
    rng = np.random.default_rng(B)
    ctx = rng.integers(0, 20, B).tolist()
    chunk = rng.choice([0, 1, 1, 3], B).tolist()
    for b, n in ((0, 40), (B // 2, 130), (B - 1, 33)):
        chunk[b] = n
    _case(ctx, chunk, 2, 1, 64, 16, seed=B)


def test_decreasing_starts_among_row_tiles_stay_in_bounds():
    import torch
    import markov_draft_sampling_amd as mds
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    T, D = 400, 64
    g = torch.Generator().manual_seed(0)
    q = torch.randn(T, 4, D, generator=g).to(torch.bfloat16).cuda()
    kp = torch.randn(8, 16, 1, D, generator=g).to(torch.bfloat16).cuda()
    table = t([[0, 1], [2, 3], [4, 5], [6, 7]])
    run = lambda starts: _run_mixed(mds, q, kp, table, t(starts))  # noqa: E731
    st, out = run([0, 300, 350, 350, 400])
    assert st == 0
    st2, out2 = run([0, 300, 20, 350, 400])  # requests 1 and 2 are out of order
    assert st2 & 8
    assert torch.equal(out2[350:], out[350:]) and torch.isfinite(out2).all()


def _run_mixed(mds, q, kp, table, starts):
    import torch
    out = torch.zeros_like(q)
    seq = torch.tensor([30, 31, 20, 32], dtype=torch.int32, device="cuda")
    ws = mds.paged_attention(q, kp, kp, table, starts, seq, out, 300, 32, causal=False)
    torch.cuda.synchronize()
    return mds.workspace_status(ws), out


@pytest.mark.parametrize("B,Hk", [(40, 8), (100, 4), (128, 3)])
def test_longest_first_order(B, Hk):
    # more work-groups than the CUs hold: requests are taken by falling length (ties, empty ones and all)
    rng = np.random.default_rng(B)
    ctx = rng.choice([0, 3, 3, 40, 77, 130], B).tolist()
    chunk = rng.choice([1, 1, 2, 0], B).tolist()
    _case(ctx, chunk, 2 * Hk, Hk, 64, 16, seed=B, idx=True)


@pytest.mark.parametrize("guess", [None, 100, 4700, 40000])
def test_some_long_sequences_among_many(guess):
    # chunks that only some requests have, a guess that is too small (the last chunk takes the rest) or too large
    rng = np.random.default_rng(1)
    ctx = rng.integers(0, 60, 40).tolist()
    ctx[3], ctx[17], ctx[30] = 10000, 4605, 4610
    chunk = rng.choice([0, 1, 2], 40).tolist()
    chunk[3], chunk[17], chunk[30] = 2, 1, 2
    _case(ctx, chunk, 16, 8, 128, 16, seed=11, idx=True, max_seq=guess)
    ctx = rng.integers(0, 700, 100).tolist()
    _case(ctx, [2] * 100, 8, 4, 64, 16, "e4m3", seed=12, max_seq=guess)


@pytest.mark.parametrize("rows", [1, 4, 20, 100])
@pytest.mark.parametrize("window", [0, 9])
def test_infinities_and_nan_stay_with_the_rows_that_see_them(rows, window):
    import torch
    import markov_draft_sampling_amd as mds
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    D, P, L = 64, 16, 200
    n = rows
    g = torch.Generator().manual_seed(rows)
    q = torch.randn(n, 2, D, generator=g).to(torch.bfloat16)
    k = torch.randn(16, P, 1, D, generator=g).to(torch.bfloat16)
    v = torch.randn(16, P, 1, D, generator=g).to(torch.bfloat16)
    kf, vf = k.view(-1, D), v.view(-1, D)
    inf, nan = float("inf"), float("nan")
    # seen by the last rows only (causal), and by the first rows only (window)
    vf[L - 1, 3], vf[L - 1, 4], vf[L - 1, 5] = inf, nan, -inf
    vf[L - 2, 3] = -inf
    kf[L - 1, 0] = nan
    vf[L - n - 8 if window else 5, 7] = inf
    kf[L - n - 8 if window else 6, 1] = 1.0
    out, lse = torch.zeros_like(q).cuda(), torch.zeros(n, 2, device="cuda")
    table = t([list(range(16))])
    mds.paged_attention(q.cuda(), k.cuda(), v.cuda(), table, t([0, n]), t([L]), out, n, L, window=window, lse=lse)
    ref, _, _, _ = sr.attention(q, k, v, table.cpu().numpy(), [0, n], [L], 1 / math.sqrt(D), True, window)
    o = out.cpu().double()
    assert torch.equal(torch.isnan(o), torch.isnan(ref))
    assert torch.equal(torch.isinf(o), torch.isinf(ref)) and torch.equal(o[torch.isinf(o)], ref[torch.isinf(ref)])
    ok = torch.isfinite(ref)
    assert ((o - ref).abs()[ok] < 2.0 ** -8 * (ref.abs()[ok] + 4.0)).all()


def test_requests_without_keys_give_zero():
    import torch
    import markov_draft_sampling_amd as mds
    # seq_lens 0 (refused), shorter than the chunk (its first tokens stand before position 0), a padding slot
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    kp = torch.randn(6, 16, 1, 64, device="cuda").to(torch.bfloat16)
    q = torch.randn(9, 2, 64, device="cuda").to(torch.bfloat16)
    out, lse = torch.full_like(q, 3.0), torch.full((9, 2), 3.0, device="cuda")
    table = t([[1, 2], [3, 4], [5, 0]])
    ws = mds.paged_attention(q, kp, kp, table, t([0, 3, 6, 9]), t([0, 2, 5]), out, 3, 32, idx_map=t([0, 1, -1]), lse=lse)
    torch.cuda.synchronize()
    assert mds.workspace_status(ws) == 0
    none = torch.tensor([1, 1, 1, 1, 0, 0, 1, 1, 1], dtype=torch.bool)
    assert (out.cpu()[none] == 0).all() and (lse.cpu()[none] == -math.inf).all()
    # token 1 of request 1 stands at position 0: it sees one key
    assert torch.equal(out[4, 0], kp[3, 0, 0]) and torch.isfinite(lse[4:6]).all()


def test_out_of_contract_device_data_is_flagged_and_stays_in_bounds():
    import torch
    import markov_draft_sampling_amd as mds
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    kp = torch.randn(4, 16, 1, 64, device="cuda").to(torch.bfloat16)
    q = torch.randn(4, 1, 64, device="cuda").to(torch.bfloat16)

    def run(table, qs, seq, idx=None, mq=4):
        out = torch.zeros_like(q)
        ws = mds.paged_attention(q, kp, kp, t(table), t(qs), t(seq), out, mq, 32, idx_map=idx)
        torch.cuda.synchronize()
        return mds.workspace_status(ws), out

    st, out = run([[1, 99]], [0, 2], [20])  # a page outside the cache: page 0 is read
    st2, out2 = run([[1, 0]], [0, 2], [20])
    assert st == 16 and st2 == 0 and torch.equal(out, out2)
    st, out = run([[1, 2]], [0, 1], [1000])  # longer than the table's row
    assert st == 8 and torch.isfinite(out).all()
    st, _ = run([[1, 2]], [0, 700], [20])  # tokens past the rows of q
    assert st & 8
    st, _ = run([[1, 2], [1, 2]], [0, 3, 1], [20, 20])  # decreasing starts
    assert st & 8
    st, out = run([[1, 2]], [0, 2], [20], idx=t([5]))  # a slot past the table
    assert st == 8 and (out == 0).all()
    st, _ = run([[1, 2]], [0, 4], [20], mq=1)  # more tokens than max_q_len: flagged when they do not fit its tiles
    assert st in (0, 8)


def test_tokens_past_max_q_len_are_flagged_and_left_alone():
    import torch
    import markov_draft_sampling_amd as mds
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator().manual_seed(5)
    kp = torch.randn((4, 16, 1, 64), generator=g).to(torch.bfloat16)
    q = torch.randn((40, 1, 64), generator=g).to(torch.bfloat16)
    out, lse = torch.full_like(q, 7.0).cuda(), torch.full((40, 1), 7.0, device="cuda")
    # one request of 40 rows where 1 was promised: its only tile has 16
    ws = mds.paged_attention(q.cuda(), kp.cuda(), kp.cuda(), t([[1, 2, 3]]), t([0, 40]), t([45]), out, 1, 64, lse=lse)
    torch.cuda.synchronize()
    assert mds.workspace_status(ws) == 8
    ref = sr.attention(q, kp.float(), kp.float(), np.array([[1, 2, 3]]), [0, 40], [45], 1 / 8)
    _check(out.cpu()[:16], lse.cpu()[:16], ref, 64, 45, 16)
    assert (out[16:] == 7.0).all() and (lse[16:] == 7.0).all()


@pytest.mark.parametrize("ctx,chunk,Hq,Hk,D", [([0, 5, 30, 100], [8] * 4, 8, 2, 64), ([3000], [1], 32, 8, 128),
                                               ([900, 20], [130, 40], 16, 8, 128), ([30] * 100, [2] * 100, 16, 8, 64)])
def test_every_row_is_written_again(ctx, chunk, Hq, Hk, D):
    # a second call writes every row and nothing else, with the same bits
    import torch
    import markov_draft_sampling_amd as mds
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator().manual_seed(len(ctx))
    seq = [a + n for a, n in zip(ctx, chunk)]
    mp = -(-max(seq) // 16)
    kp = torch.randn((len(ctx) * mp, 16, Hk, D), generator=g).to(torch.bfloat16).cuda()
    table = torch.arange(len(ctx) * mp, dtype=torch.int32, device="cuda").view(-1, mp)
    T = sum(chunk)
    q = torch.randn((T + 3, Hq, D), generator=g).to(torch.bfloat16).cuda()
    got = []
    ws = None
    for fill in (7.0, -3.0):
        out, lse = torch.full_like(q, fill), torch.full((T + 3, Hq), fill, device="cuda")
        ws = mds.paged_attention(q, kp, kp, table, t(np.cumsum([0] + chunk)), t(seq), out, max(chunk), max(seq), lse=lse,
                                 workspace=ws)
        assert (out[T:] == fill).all() and (lse[T:] == fill).all()
        got.append((out[:T], lse[:T]))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("Hq,Hk,D", [(256, 1, 64), (200, 1, 128), (64, 64, 64), (130, 2, 64)])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_many_heads(Hq, Hk, D, cache):
    # one token's heads over more than one row tile, and a key head for each
    _case([50, 0, 333], [2, 1, 1], Hq, Hk, D, 16, cache, seed=Hq)


def test_two_calls_at_once_on_two_streams():
    import torch
    import markov_draft_sampling_amd as mds
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator().manual_seed(3)
    kp = torch.randn((400, 16, 2, 128), generator=g).to(torch.bfloat16).cuda()
    q = [torch.randn((n, 8, 128), generator=g).to(torch.bfloat16).cuda() for n in (300, 9)]
    table = t(np.random.default_rng(0).permutation(400)[:384].reshape(3, 128))
    qs, seq = [t([0, 200, 250, 300]), t([0, 8, 8, 9])], t([1900, 700, 2040])
    mq, ms = (200, 8), 2048
    want = []
    for i in range(2):
        want.append(torch.zeros_like(q[i]))
        mds.paged_attention(q[i], kp, kp, table, qs[i], seq, want[i], mq[i], ms)
    got = [torch.zeros_like(x) for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(4):
        for i, st in enumerate(streams):
            mds.paged_attention(q[i], kp, kp, table, qs[i], seq, got[i], mq[i], ms, stream=st)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i], want[i])


@pytest.mark.parametrize("B", [70, 140])
@pytest.mark.parametrize("D,cache", [(64, "bf16"), (128, "bf16"), (64, "e4m3"), (128, "e4m3")])
@pytest.mark.parametrize("G", [2, 7])
def test_many_short_sequences(B, D, cache, G):
    # fewer key groups a work-group: more tiles than CUs over short sequences
    rng = np.random.default_rng(B)
    ctx = rng.integers(0, 470, B).tolist()
    _case(ctx, rng.choice([1, 2, 3, 4], B).tolist(), 4 * G, 4, D, 16, cache, seed=B, idx=True,
          window=0 if G == 2 else 300)


@pytest.mark.parametrize("D,cache", [(64, "bf16"), (128, "bf16"), (64, "e4m3"), (128, "e4m3")])
def test_64_row_tiles_by_work_groups(D, cache):
    # two key groups: more work-groups than CUs; one: many requests over short sequences
    rng = np.random.default_rng(D)
    ctx = rng.integers(0, 300, 130).tolist()
    chunk = rng.choice([5, 8, 0, 7], 130).tolist()
    _case(ctx, chunk, 64, 8, D, 16, cache, seed=1, idx=True)
    _case(ctx[:45], chunk[:45], 64, 8, D, 16, cache, seed=2, max_seq=2000, window=100)
    _case([0, 60], [150, 77], 64, 32, D, 32, cache, seed=3, max_seq=1100)
    _case([9, 60], [150, 77], 64, 32, D, 16, cache, seed=4, max_seq=1100, causal=False)
    _case([900, 60], [150, 77], 64, 32, D, 16, cache, seed=5, window=400, max_q=1200, max_seq=1100)


# guesses of the longest sequence that lead to tiles of 64 and 128 rows for prompts as short as these
TALL = {64: 1100, 128: 600000}


@pytest.mark.parametrize("rows", sorted(TALL))
@pytest.mark.parametrize("D,cache", [(64, "bf16"), (128, "bf16"), (64, "e4m3"), (128, "e4m3")])
def test_tall_tiles(rows, D, cache):
    _case([0, 40, 130], [150, 1, 77], 4, 2, D, 16, cache, seed=9, q_layout="htd", max_seq=TALL[rows])
    _case([100], [130], 3, 1, D, 32, cache, window=50, seed=1, max_seq=TALL[rows], max_q=TALL[rows])
    _case([100, 7], [130, 200], 3, 1, D, 16, cache, causal=False, seed=2, max_seq=TALL[rows], idx=True)
    _case([0], [300], 1, 1, D, 64, cache, window=1, seed=3, max_seq=TALL[rows], max_q=TALL[rows], layout="hnd")


def test_tall_tiles_over_split_keys():
    # chunks of 1536 and of 1152 keys of 128-row tiles, of 1152 of 64-row tiles; some of them a row does not reach
    _case([4000], [300], 64, 32, 64, 16, seed=4)
    _case([2100], [100], 256, 64, 64, 16, "e4m3", seed=5, window=2000)
    _case([2100], [100], 8, 2, 128, 16, seed=6, window=2000)


@pytest.mark.parametrize("tall", sorted(TALL))
@pytest.mark.parametrize("D", [64, 128])
def test_infinities_and_nan_in_tall_tiles(tall, D):
    import torch
    import markov_draft_sampling_amd as mds
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    L, n, window = 400, 190, 30
    g = torch.Generator().manual_seed(tall)
    q = torch.randn(n, 2, D, generator=g).to(torch.bfloat16)
    k = torch.randn(25, 16, 1, D, generator=g).to(torch.bfloat16)
    v = torch.randn(25, 16, 1, D, generator=g).to(torch.bfloat16)
    kf, vf = k.view(-1, D), v.view(-1, D)
    inf, nan = float("inf"), float("nan")
    vf[L - 1, 3], vf[L - 1, 4], vf[L - 1, 5] = inf, nan, -inf
    vf[300, 7], vf[301, 7], vf[250, 9] = inf, -inf, nan
    kf[L - 2, 0], kf[320, 1] = nan, nan
    out = torch.zeros_like(q).cuda()
    table = t([list(range(25))])
    mds.paged_attention(q.cuda(), k.cuda(), v.cuda(), table, t([0, n]), t([L]), out, TALL[tall], TALL[tall],
                        window=window)
    ref, _, _, _ = sr.attention(q, k, v, table.cpu().numpy(), [0, n], [L], 1 / math.sqrt(D), True, window)
    o = out.cpu().double()
    assert torch.equal(torch.isnan(o), torch.isnan(ref))
    assert torch.equal(torch.isinf(o), torch.isinf(ref)) and torch.equal(o[torch.isinf(o)], ref[torch.isinf(ref)])
    ok = torch.isfinite(ref)
    assert ok.any() and ((o - ref).abs()[ok] < 2.0 ** -8 * (ref.abs()[ok] + 4.0)).all()


def test_large_scores_and_a_peak_late_in_the_row():
    # scores up to some hundreds: the running maximum has to move many times
    _case([700], [4], 2, 1, 128, 16, seed=8, scale=2.0, qgain=3.0)


@pytest.mark.parametrize("D,window", [(64, 0), (128, 0), (128, 700)])
def test_one_workspace_for_the_largest_step_and_smaller_ones(D, window):
    import torch
    import markov_draft_sampling_amd as mds
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    rng = np.random.default_rng(D)
    T, B, Hq, Hk, mq, ms = 300, 8, 16, 4, 200, 6000
    ws = mds.new_workspace(mds.paged_attention_workspace_bytes(T, B, Hq, Hk, D, mq, ms, window))
    kp = torch.randn((400, 16, Hk, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    table = t(rng.integers(0, 400, (B, 375)))
    for chunk in ([200, 40, 8, 8, 8, 8, 8, 8], [8] * 8, [1] * 8, [1], [8], [17, 3], [130], [64, 1, 1], [1, 0, 5, 2, 2, 2, 1]):
        for longest in (ms, 900, 300):
            n, b = sum(chunk), len(chunk)
            seq = [int(x) for x in rng.integers(longest // 2, longest + 1, b)]
            q = torch.randn((n, Hq, D), device="cuda").to(torch.bfloat16)
            args = (q, kp, kp, table[:b], t(np.cumsum([0] + chunk)), t(seq))
            want, got = torch.zeros_like(q), torch.full_like(q, 7.0)
            mds.paged_attention(*args, want, max(chunk), longest, window=window)
            mds.paged_attention(*args, got, max(chunk), longest, window=window, workspace=ws)
            assert torch.equal(got, want), (chunk, longest)
    assert mds.workspace_status(ws) == 0


def test_a_new_workspace_in_used_memory_has_no_status_and_no_other_clearing():
    import torch
    import markov_draft_sampling_amd as mds
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    kp = torch.randn(300, 16, 2, 64, device="cuda").to(torch.bfloat16)
    q = torch.randn(3, 4, 64, device="cuda").to(torch.bfloat16)
    table, qs, seq = torch.arange(300, dtype=torch.int32, device="cuda").view(1, 300), t([0, 3]), t([4000])
    n = mds.paged_attention_workspace_bytes(3, 1, 4, 2, 64, 3, 4000)
    want, got = torch.zeros_like(q), torch.zeros_like(q)
    mds.paged_attention(q, kp, kp, table, qs, seq, want, 3, 4000,
                        workspace=torch.zeros(n, dtype=torch.uint8, device="cuda"))
    dirty = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    mds.paged_attention(q, kp, kp, table, qs, seq, got, 3, 4000, workspace=dirty)
    dirty.fill_(255)
    at = dirty.data_ptr()
    del dirty
    again = torch.zeros_like(q)
    ws = mds.paged_attention(q, kp, kp, table, qs, seq, again, 3, 4000)
    assert torch.equal(got, want) and torch.equal(again, want) and mds.workspace_status(ws) == 0
    # two key heads of one 16-row tile: rows past the request's are nobody's, and stay as the memory was
    assert ws.data_ptr() != at or (ws == 255).any()


def test_strides_of_dimensions_of_one():
    # one token, one head, one page: torch gives such dimensions whatever stride the view was made with
    import torch
    import markov_draft_sampling_amd as mds
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    D = 64
    odd = lambda x: x.as_strided(x.shape, [3 if n == 1 else s for n, s in zip(x.shape, x.stride())])  # noqa: E731
    kv = torch.randn(1, 1, D, device="cuda").to(torch.bfloat16)
    q = torch.randn(1, 1, D, device="cuda").to(torch.bfloat16)
    slot = torch.tensor([5], dtype=torch.int64, device="cuda")
    got = []
    for view in (lambda x: x, odd):
        pages = torch.ones(1, 16, 1, D, device="cuda", dtype=torch.bfloat16)
        mds.kv_append(view(kv), view(kv), view(pages), view(pages.clone()), slot)
        out = torch.zeros_like(q)
        mds.paged_attention(view(q), view(pages), view(pages), t([[0]]), t([0, 1]), t([6]), view(out), 1, 6)
        got.append((pages, out))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert torch.equal(got[1][0][0, 5, 0], kv[0, 0])


def test_offsets_past_32_bits():
    # pages whose offset passes 2^31 bytes and 2^31 elements: a strided view over a large buffer
    import torch
    import markov_draft_sampling_amd as mds
    P, D, stride = 16, 64, 1 << 30  # elements from page to page
    big = torch.zeros(4 * stride, dtype=torch.bfloat16, device="cuda")
    kp = big.as_strided((4, P, 1, D), (stride, D, D, 1))
    small = torch.randn(4, P, 1, D, device="cuda").to(torch.bfloat16)
    kp.copy_(small)
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn(2, 2, D, device="cuda").to(torch.bfloat16)
    outs = []
    for pages in (kp, small):
        out = torch.zeros_like(q)
        mds.paged_attention(q, pages, pages, t([[3, 1, 2, 0]]), t([0, 2]), t([60]), out, 2, 64)
        outs.append(out)
    assert torch.equal(*outs)
    slots = torch.tensor([3 * P + 5, 1], dtype=torch.int64, device="cuda")
    kv = torch.randn(2, 1, D, device="cuda").to(torch.bfloat16)
    mds.kv_append(kv, kv, kp, kp.clone(), slots)
    assert torch.equal(kp[3, 5], kv[0]) and torch.equal(kp[0, 1], kv[1])


def test_graph_replays_and_a_side_stream():
    import torch
    import markov_draft_sampling_amd as mds
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    g0 = torch.Generator().manual_seed(1)
    kp = torch.randn((300, 16, 2, 128), generator=g0).to(torch.bfloat16).cuda()
    q = torch.randn((16, 8, 128), generator=g0).to(torch.bfloat16).cuda()
    table = t(np.random.default_rng(0).permutation(300)[:256].reshape(2, 128))
    qs, seq = t([0, 8, 16]), t([2000, 100])
    out, lse = torch.zeros_like(q), torch.zeros(16, 8, device="cuda")
    ws = mds.new_workspace(mds.paged_attention_workspace_bytes(16, 2, 8, 2, 128, 8, 2048))
    call = lambda o: mds.paged_attention(q, kp, kp, table, qs, seq, o, 8, 2048, lse=lse, workspace=ws)  # noqa: E731
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    for i in range(5):
        seq.copy_(t([2000 - 300 * i, 100 + i]))
        q.copy_(torch.randn((16, 8, 128), generator=g0).to(torch.bfloat16).cuda())
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        want = torch.zeros_like(q)
        mds.paged_attention(q, kp, kp, table, qs, seq, want, 8, 2048)
        assert torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = torch.zeros_like(q)
    side.wait_stream(torch.cuda.current_stream())
    mds.paged_attention(q, kp, kp, table, qs, seq, got, 8, 2048, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_refuses_mismatched_tensors():
    import torch
    import markov_draft_sampling_amd as mds
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    kp = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device="cuda")
    ok = dict(q=q, k=kp, v=kp, table=t([[0, 1]]), qs=t([0, 4]), seq=t([4]), out=torch.zeros_like(q))

    def run(**kw):
        a = {**ok, **{k: v for k, v in kw.items() if k in ok}}
        extra = {k: v for k, v in kw.items() if k not in ok}
        mds.paged_attention(a["q"], a["k"], a["v"], a["table"], a["qs"], a["seq"], a["out"], 4, 4, **extra)

    run()
    for bad in (dict(q=q.half()), dict(q=q.cpu()), dict(v=kp[:1]), dict(table=t([0, 1])), dict(qs=t([0])),
                dict(seq=t([4]).long()), dict(out=torch.zeros(4, 4, 32, dtype=torch.bfloat16, device="cuda")),
                dict(k=kp.half(), v=kp.half()), dict(lse=torch.zeros(3, device="cuda")), dict(idx_map=t([0, 0])),
                dict(k_scale=torch.ones(2, device="cuda")), dict(scale=-1.0), dict(window=-3),
                dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(mds.MdsError):
            run(**bad)
