"""Attention with a window and first tokens that stay visible, on the GPU
against float64 within the bounds of its roundings. Every page of which a
request's tokens see no key holds NaN, and its entries of the block table are
no pages at all."""
from __future__ import annotations

import math

import numpy as np
import pytest

import layer_ref as lr
import serving_ref as sr

pytestmark = pytest.mark.gpu


def _case(ctx, chunk, Hq, Hk, D, P, window, sinks, cache="bf16", causal=True, pad=2, seed=0, idx=False, max_q=None,
          max_seq=None, layout="nhd", nan_values=False, huge=False):
    import torch
    import markov_draft_sampling_amd as mds
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    B = len(ctx)
    seq = [a + n for a, n in zip(ctx, chunk)]
    held = [max(1, -(-x // P)) for x in seq]
    NP = sum(held) + 2
    pages = rng.permutation(NP - 1) + 1  # page 0 belongs to nobody
    MP = max(held) + 1
    n_slots = B + 3 if idx else B
    slots = rng.permutation(n_slots)[:B] if idx else np.arange(B)
    table = np.full((n_slots, MP), 1 << 30, np.int32)
    at = 0
    for b in range(B):
        table[slots[b], :held[b]] = pages[at:at + held[b]]
        at += held[b]
    T = sum(chunk)
    q = (torch.randn((T + pad, Hq, D), generator=g) * 1.5).to(torch.bfloat16)
    kv = []
    for _ in range(2):
        x = torch.randn((NP, P, Hk, D), generator=g)
        kv.append((x * 60).clamp(-448, 448).to(torch.float8_e4m3fn) if cache == "e4m3" else x.to(torch.bfloat16))
    ks = vs = None
    if cache == "e4m3":
        ks, vs = (torch.tensor(rng.uniform(0.9, 1.1, Hk) / 60, dtype=torch.float32) for _ in range(2))
    qs = np.concatenate([[0], np.cumsum(chunk)]).astype(np.int32)
    scale = 1 / math.sqrt(D)
    *ref, seen = lr.attention_sinks(q[:T], kv[0].float(), kv[1].float(), table, qs, seq, scale, causal, window, sinks,
                                    slots if idx else None, ks, vs)
    # what nobody sees: pages of NaN, entries that are no pages
    raw = torch.uint8 if cache == "e4m3" else torch.int16
    nan = 0x7F if cache == "e4m3" else 0x7FC0
    dev, used = [], {int(table[slots[b]][p]) for b in range(B) for p in seen[b]}
    for x in kv:
        d = x.clone()
        for p in range(NP):
            if p not in used:
                d.view(raw)[p] = nan
        for b in range(B):  # behind a sequence's end in its last page
            for p in range(seq[b], held[b] * P):
                if p // P in seen[b]:
                    d.view(raw)[table[slots[b]][p // P], p % P] = nan
        d = d.cuda()
        if layout == "hnd":
            d = d.view(raw).transpose(1, 2).contiguous().transpose(1, 2).view(d.dtype)
        dev.append(d)
    tab = table.copy()
    for b in range(B):
        for p in range(MP):
            if p not in seen[b]:
                tab[slots[b], p] = (1 << 30) if p % 2 else -5
    if nan_values:  # of one key between the first tokens and the window, in a page that is read
        assert B == 1 and nan_values < seq[0]
        dev[1].view(raw)[table[0][nan_values // P], nan_values % P] = nan
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full((T + pad, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + pad, Hq), 7.0, device="cuda")
    args = dict(causal=causal, window=window, sinks=sinks, idx_map=t(slots) if idx else None, lse=lse,
                k_scale=None if ks is None else ks.cuda(), v_scale=None if vs is None else vs.cuda())
    mq, ms = max(chunk) if max_q is None else max_q, max(seq) if max_seq is None else max_seq
    print(f"sinks ctx {list(ctx)[:6]} chunk {list(chunk)[:6]} Hq {Hq} Hk {Hk} D {D} P {P} {cache} causal {causal} "
          f"window {window} sinks {sinks}", flush=True)
    call = (q.cuda(), dev[0], dev[1], t(tab), t(qs), t(seq), out, mq, ms)
    ws = mds.paged_attention(*call, **args)
    torch.cuda.synchronize()
    assert mds.workspace_status(ws) == 0
    again = out.clone()
    mds.paged_attention(*call, workspace=ws, **args)
    assert torch.equal(again, out)
    o, z = out.cpu(), lse.cpu()
    assert (o[T:] == 7).all() and (z[T:] == 7).all()
    r, rl, A, S = ref
    tol, ltol = sr.attention_tolerance(r, A, S, D, max(seq))
    err = (o[:T].double() - r).abs()
    assert (err <= tol).all(), (float((err / tol).max()), torch.nonzero(~(err <= tol))[:4].tolist())
    none = rl == -math.inf
    assert (z[:T][none] == -math.inf).all() and (o[:T][none] == 0).all()
    assert ((z[:T].double() - rl).abs()[~none] <= ltol[~none]).all()
    return o, z


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(1, 1), (17, 4), (64, 64), (100, 63), (300, 65), (1000, 200), (40, 5000)])
def test_one_token(window, sinks, cache, D):
    _case([0, 1, 5, 63, 64, 130, 700, 2047], [1] * 8, 6, 2, D, 16, window, sinks, cache, seed=window)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hk,chunk", [(4, 4, 8), (8, 2, 8), (16, 1, 8), (16, 2, 20), (32, 1, 17)])
@pytest.mark.parametrize("window,sinks", [(5, 1), (64, 4), (129, 70), (513, 16)])
def test_chunks_of_every_tile_height(window, sinks, Hq, Hk, chunk, cache):
    # 8 to 544 rows a key head
    _case([0, 3, 200, 900, 77], [chunk, 0, chunk, chunk - 1, 1], Hq, Hk, 64, 32, window, sinks, cache, seed=chunk)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(3, 2), (128, 4), (200, 130), (5000, 4)])
def test_prompts(window, sinks, D):
    _case([0, 600], [333, 150], 4, 2, D, 16, window, sinks, seed=1)


@pytest.mark.parametrize("P", [16, 32, 64, 128, 1024])
def test_page_sizes_and_layouts(P):
    _case([2100, 40, 1500], [3, 4, 8], 4, 2, 128, P, 90, 20, layout="hnd", idx=True)
    _case([2100, 40, 1500], [3, 4, 8], 4, 2, 64, P, 90, 20, cache="e4m3", idx=True)


@pytest.mark.parametrize("window,sinks", [(8, 3), (64, 64), (65, 1)])
def test_a_block_that_sees_both_ways(window, sinks):
    _case([0, 130, 1000], [7, 7, 7], 8, 2, 64, 16, window, sinks, causal=False)


@pytest.mark.parametrize("batch,ctx", [(1, 30000), (3, 9000), (130, 300)])
def test_split_keys(batch, ctx):
    rng = np.random.default_rng(batch)
    lens = rng.integers(ctx // 2, ctx, batch).tolist()
    _case(lens, [1] * batch, 2, 1, 128, 64, ctx // 3, 100, seed=batch)
    _case(lens, [2] * batch, 2, 1, 64, 64, ctx // 4, 5, cache="e4m3", seed=batch, max_seq=40 * ctx)
    _case(lens, [1] * batch, 2, 1, 64, 64, ctx // 4, 5, seed=batch, max_seq=10)  # a guess that is too short


def test_prompts_over_128_rows_and_split():
    _case([5000], [700], 8, 2, 128, 16, 4500, 33)
    _case([300, 2000], [600, 520], 16, 1, 64, 16, 700, 64, seed=3)


def test_a_prompt_beside_single_tokens():
    # tiles numbered by their rows instead of by request
    _case([3000] + list(range(10, 1000, 50)), [260] + [1] * 20, 4, 2, 64, 16, 200, 20, idx=True)
    _case(list(range(10, 1000, 50)) + [900], [0, 3] * 10 + [150], 8, 2, 128, 32, 100, 70, cache="e4m3")


def test_more_work_groups_than_cus_longest_first():
    rng = np.random.default_rng(0)
    lens = rng.integers(1, 7000, 70).tolist()
    _case(lens, [1] * 70, 4, 4, 64, 64, 5000, 10, seed=5)
    _case(lens, [2] * 70, 8, 4, 64, 64, 5000, 10, cache="e4m3", seed=6, idx=True)


def test_pages_past_32_bits():
    import torch
    import markov_draft_sampling_amd as mds
    NP, P, H, D = 140000, 16, 8, 128  # 32 KB a page: the last one is 4.6 GB in
    kp, vp = (torch.zeros((NP, P, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(0)
    mine = [NP - 1, 5, NP - 70, 70000]
    k, v = (torch.randn((64, H, D), generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((64, H, D), generator=g).to(torch.bfloat16)
    slot = torch.tensor([mine[i // P] * P + i % P for i in range(64)], device="cuda")
    pos, qo = torch.zeros(64, dtype=torch.int64, device="cuda"), torch.zeros((64, H, D), dtype=torch.bfloat16, device="cuda")
    mds.qk_norm_rope_append(q.cuda(), k.cuda(), v.cuda(), pos, None, qo, kp, vp, slot)
    assert torch.equal(qo.cpu(), q) and torch.equal(kp[mine].cpu().view(64, H, D), k) and torch.equal(vp[mine].cpu().view(64, H, D), v)
    assert int((kp != 0).any(-1).any(-1).sum()) == 64
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.zeros((1, H, D), dtype=torch.bfloat16, device="cuda")
    mds.paged_attention(qo[:1], kp, vp, t([mine]), t([0, 1]), t([63]), out, 1, 63, window=20, sinks=3)
    r, _, A, S, _ = lr.attention_sinks(q[:1], k.float().view(4, P, H, D), v.float().view(4, P, H, D), [[0, 1, 2, 3]], [0, 1],
                                       [63], 1 / math.sqrt(D), True, 20, 3)
    tol, _ = sr.attention_tolerance(r, A, S, D, 63)
    assert ((out.cpu().double() - r).abs() <= tol).all()


def test_the_edges_of_both_parts():
    # every distance of the window from the first tokens, over two blocks of 64 keys
    for ctx in range(60, 200, 7):
        _case([ctx], [3], 2, 1, 64, 16, 33, 20, seed=ctx)
    for sinks in (15, 16, 17, 31, 33, 47, 48, 63, 64, 65, 127, 129):
        _case([400, 140], [2, 5], 2, 1, 64, 16, 50, sinks, seed=sinks)


def test_nan_between_the_two_parts_reaches_nobody():
    # first tokens 0 .. 3 and the window from 37 on share no page with key 20, but key 10 shares one with the first tokens
    _case([60], [1], 2, 1, 64, 16, 24, 4, nan_values=10)
    _case([60], [1], 2, 1, 64, 16, 24, 4, nan_values=35)
    _case([1000], [5], 4, 1, 128, 64, 100, 4, nan_values=30)


def test_an_infinite_value_of_a_first_token_reaches_all():
    import torch
    import markov_draft_sampling_amd as mds
    g = torch.Generator().manual_seed(0)
    kp, vp = (torch.randn((20, 16, 1, 64), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    vp[0, 2, 0, 5] = float("inf")
    vp[15, 0, 0, 9] = float("inf")  # key 240, which only some tokens of the chunk see
    q = torch.randn((30, 2, 64), generator=g).to(torch.bfloat16).cuda()
    out = torch.zeros_like(q)
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    mds.paged_attention(q, kp, vp, t([list(range(20))]), t([0, 30]), t([290]), out, 30, 290, window=30, sinks=3)
    o = out.float().cpu()
    assert (o[:, :, 5] == math.inf).all()
    sees = torch.tensor([240 <= 260 + i and 240 > 260 + i - 30 for i in range(30)])
    assert (o[sees][:, :, 9] == math.inf).all() and o[~sees][:, :, 9].isfinite().all()
    assert o[:, :, [i for i in range(64) if i not in (5, 9)]].isfinite().all()


def test_without_a_window_or_first_tokens_it_is_the_call_without():
    import torch
    import markov_draft_sampling_amd as mds
    g = torch.Generator().manual_seed(0)
    kp, vp = (torch.randn((40, 16, 2, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn((16, 4, 128), generator=g).to(torch.bfloat16).cuda()
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.randperm(40, generator=g).view(2, 20).int().cuda()
    call = (q, kp, vp, table, t([0, 8, 16]), t([300, 317]))
    outs = []
    for kw in (dict(), dict(sinks=7), dict(window=400), dict(sinks=7, window=400)):
        outs.append(torch.zeros_like(q))
        mds.paged_attention(*call, outs[-1], 8, 317, **kw)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    # a window that holds every key: the work may be cut another way, which moves the maximum that a probability is taken
    # against before it is rounded: each of the two is within 2^-8 of the value and 2^-8 of sum p |v| <= max |v| off
    r = outs[0].double()
    assert ((outs[3].double() - r).abs() <= 2.01 * (2.0 ** -8 * r.abs() + 2.0 ** -8 * vp.abs().max().double())).all()
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    mds.paged_attention(*call, a, 8, 317, window=50)
    mds.paged_attention(*call, b, 8, 317, window=50, sinks=0)
    assert torch.equal(a, b)


def test_padding_requests_and_requests_of_nothing():
    import torch
    import markov_draft_sampling_amd as mds
    g = torch.Generator().manual_seed(0)
    kp, vp = (torch.randn((20, 16, 1, 64), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn((6, 2, 64), generator=g).to(torch.bfloat16).cuda()
    out, lse = torch.full_like(q, 7.0), torch.full((6, 2), 7.0, device="cuda")
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.arange(20).view(2, 10).int().cuda()
    ws = mds.paged_attention(q, kp, vp, table, t([0, 2, 2, 4, 5]), t([150, 30, 150, 0]), out, 2, 150, window=20, sinks=4,
                             idx_map=t([1, 0, -1, 0]), lse=lse)
    o, z = out.cpu(), lse.cpu()
    assert mds.workspace_status(ws) == 0
    assert (o[2:5] == 0).all() and (z[2:5] == -math.inf).all()
    assert (o[5:] == 7).all() and (z[5:] == 7).all()
    assert o[:2].isfinite().all() and z[:2].isfinite().all()


def test_one_workspace_two_calls_at_once_and_a_graph():
    import torch
    import markov_draft_sampling_amd as mds
    g = torch.Generator().manual_seed(0)
    B, P = 8, 16
    kp, vp = (torch.randn((8 * 130, P, 2, 128), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    table = torch.randperm(8 * 130, generator=g).view(8, 130).int().cuda()
    q = torch.randn((B, 8, 128), generator=g).to(torch.bfloat16).cuda()
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    seq, qs = t([2000, 1, 300, 64, 1999, 700, 5, 1200]), t(list(range(B + 1)))
    size = mds.paged_attention_workspace_bytes(B, B, 8, 2, 128, 1, 2080, 1500, 8)
    ws = [mds.new_workspace(size) for _ in range(2)]
    out, want = torch.zeros_like(q), torch.zeros_like(q)
    call = lambda o, w, s=None: mds.paged_attention(q, kp, vp, table, qs, seq, o, 1, 2080, window=1500,  # noqa: E731
                                                    sinks=8, workspace=w, stream=s)
    call(want, ws[0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = torch.zeros_like(q)
    call(out, ws[0])
    call(other, ws[1], side)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws[0])
    for i in range(4):
        seq.add_(torch.tensor([3, 100, 1, 0, 7, 500, 64, 1], dtype=torch.int32).cuda())
        q.mul_(1.1)
        graph.replay()
        call(want, ws[1])
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
