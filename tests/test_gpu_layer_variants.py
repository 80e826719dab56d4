"""Every variant of the kernels of a layer's step that a call can take, on the
GPU, at remainders of its tiles (the sizes: layer_cases.py)."""
from __future__ import annotations

import math

import numpy as np
import pytest

import layer_cases as lc
import layer_ref as lr
import serving_ref as sr
from test_gpu_attention_sinks import _case
from test_gpu_rope import _check, _expected, _inputs, _pages

pytestmark = pytest.mark.gpu


def _mx_matrix(V, H, seed):
    """(float64 weights, tiled codes, tiled scales), all on the GPU."""
    import torch
    import markov_draft_sampling_amd as mds
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (V, H // 2), generator=g, dtype=torch.uint8, device="cuda")
    scales = torch.randint(117, 124, (V, H // 32), generator=g, dtype=torch.uint8, device="cuda")
    value = torch.from_numpy(lr.E2M1).cuda()
    w = torch.stack([value[(codes & 15).long()], value[(codes >> 4).long()]], -1).view(V, H // 32, 32)
    w = (w * torch.exp2(scales.double() - 127)[..., None]).view(V, H)
    return w, *mds.tile_lm_head_mxfp4(codes, scales)


@pytest.mark.parametrize("V,some", lc.MXFP4_HEAD)
def test_lm_head(V, some):
    # five tiles of columns, the last word of scales short. Bounds of float32 sums as in test_gpu_lm_head_mxfp4.py: products
    # exact, H / 32 matrix instructions with at most two roundings or truncations of a partial sum (2^-23 each), four sums
    # joined; the float64 products' own error is 2^-29 of that.
    import torch
    import markov_draft_sampling_amd as mds
    H = 640
    w, tiled, ts = _mx_matrix(V, H, V)
    wt, wa = w.T.contiguous(), w.abs().T.contiguous()
    for i, rows in enumerate(some):
        K = next((k for k in (8, 7, 5, 3) if rows % k == 0), 1)
        pad, bf16 = (V % 4 + i) % 5, i % 3 == 2
        print(f"4-bit LM head rows {rows} (K {K}) V {V} pad {pad} bf16 {bf16}", flush=True)
        g = torch.Generator().manual_seed(rows)
        x = torch.full((rows, H + 8), float("nan"), dtype=torch.bfloat16)
        x[:, :H] = torch.randn((rows, H), generator=g).to(torch.bfloat16)
        n = rows - (rows > 1)
        x[n:, 77] = float("nan")  # of the last of several rows: reaches its own logits alone
        x = x.cuda()
        out = torch.full((rows // K, K + i % 2, V + pad), 7.25, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
        mds.lm_head_mxfp4(x[:, :H], tiled, ts, out[..., :V], K)
        again = out.clone()
        mds.lm_head_mxfp4(x[:, :H], tiled, ts, out[..., :V], K)
        raw = torch.int16 if bf16 else torch.int32
        assert torch.equal(again.view(raw), out.view(raw))
        assert (out[:, K:] == 7.25).all() and (out[..., V:] == 7.25).all()
        got = out[:, :K, :V].reshape(rows, V)
        assert got[n:].isnan().all()
        xd = x[:n, :H].double()
        z, a = xd @ wt, xd.abs() @ wa
        tol = (4 * H / 32 + 16) * 2.0 ** -24 * a + 1e-37
        if bf16:
            tol += 2.0 ** -8 * (z.abs() + tol)
        err = (got[:n].double() - z).abs()
        assert (err <= tol).all(), (float((err / tol).max()), torch.nonzero(~(err <= tol))[:4].tolist())


@pytest.mark.parametrize("T,Hq,Hk,D,R,interleaved,norm,to,short", lc.ROPE)
def test_rotation(T, Hq, Hk, D, R, interleaved, norm, to, short):
    import torch
    import markov_draft_sampling_amd as mds
    s = _inputs(T, Hq, Hk, D, R, norm, seed=T)
    args = dict(q_weight=s["qw"], k_weight=s["kw"], interleaved=interleaved, rope_scale=1.1)
    (rq, eq), (rk, ek) = _expected(s, 1.1, interleaved)
    qo = torch.full((T + 2, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    parts = [slice(t, min(t + short, T)) for t in range(0, T, short)]
    print(f"rotation T {T} heads {Hq}/{Hk} D {D} R {R} to {to}", flush=True)
    if to == "rows":
        ko = torch.full((T + 2, Hk, D), 7.0, dtype=torch.bfloat16, device="cuda")
        mds.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], qo[:T], ko[:T], **args)
        _check(qo[:T], rq, eq)
        _check(ko[:T], rk, ek)
        assert (qo[T:] == 7).all() and (ko[T:] == 7).all()
        q2, k2 = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        for p in parts:
            mds.qk_norm_rope(s["q"][p], s["k"][p], s["pos"][p], s["freq"], q2[p], k2[p], **args)
        assert torch.equal(q2, qo[:T]) and torch.equal(k2, ko[:T])
        mds.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], s["q"], s["k"], **args)  # over its own input
        assert torch.equal(s["q"], qo[:T]) and torch.equal(s["k"], ko[:T])
        return
    rng = np.random.default_rng(T)
    P, NP = 32, -(-T // 32) + 2
    slot = rng.permutation(NP * P)[:T].astype(np.int64)
    slot[5], slot[T - 1], slot[T // 2] = -1, -9, NP * P  # two of padding, one past the cache
    live = (slot >= 0) & (slot < NP * P)
    ks = vs = None
    if to == "e4m3":
        ks, vs = (torch.tensor(rng.uniform(0.002, 0.03, Hk), dtype=torch.float32).cuda() for _ in range(2))
    kp, vp = _pages(NP, P, Hk, D, to, "hnd", 1), _pages(NP, P, Hk, D, to, "nhd", 2)
    k2, v2, q2 = kp.clone(), vp.clone(), torch.empty_like(s["q"])
    raw = lambda t: t.view(torch.uint8 if to == "e4m3" else torch.int16)  # noqa: E731
    k0, v0 = raw(kp).cpu().reshape(NP * P, Hk, D), raw(vp).cpu().reshape(NP * P, Hk, D)
    sl = torch.from_numpy(slot).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mds.qk_norm_rope_append(s["q"], s["k"], s["v"], s["pos"], s["freq"], qo[:T], kp, vp, sl, k_scale=ks, v_scale=vs,
                            status=status, **args)
    assert int(status.item()) == mds.STATUS_BAD_PAGE
    for p in parts:
        mds.qk_norm_rope_append(s["q"][p], s["k"][p], s["v"][p], s["pos"][p], s["freq"], q2[p], k2, v2, sl[p], k_scale=ks,
                                v_scale=vs, status=status, **args)
    assert torch.equal(q2, qo[:T]) and torch.equal(raw(k2), raw(kp)) and torch.equal(raw(v2), raw(vp))
    _check(qo[:T], rq, eq)  # of every token, those without a slot too
    assert (qo[T:] == 7).all()
    rest = np.setdiff1d(np.arange(NP * P), slot[live])
    assert torch.equal(raw(kp).cpu().reshape(NP * P, Hk, D)[rest], k0[rest])
    assert torch.equal(raw(vp).cpu().reshape(NP * P, Hk, D)[rest], v0[rest])
    k, v = (x.float().cpu().reshape(NP * P, Hk, D)[slot[live]] for x in (kp, vp))
    rk, ek, x = rk[live], ek[live], s["v"].cpu().float()[live]
    if to == "bf16":
        _check(k, rk, ek)
        assert torch.equal(v, x)
        return
    # rounded once: half a step of a code (2^-4, or 2^-10 below the normal ones) on what float32 leaves of y / scale,
    # as in test_gpu_rope.py
    assert np.array_equal(v.numpy(), sr.e4m3_round((x / vs.cpu()[:, None]).numpy()))
    sc = ks.cpu().double()[:, None]
    z, fuzz = (rk / sc).clamp(-448, 448), (ek / sc + 2.0 ** -23 * (rk / sc).abs()) * 1.01
    tol = torch.maximum(2.0 ** -4 * (z.abs() + fuzz), torch.tensor(2.0 ** -10)) + fuzz
    assert ((k.double() - z).abs() <= tol).all()
    lo, hi = sr.e4m3_round((z - fuzz).float().numpy()), sr.e4m3_round((z + fuzz).float().numpy())
    sure = lo == hi
    assert sure.mean() > 0.99 and (k.double().numpy()[sure] == lo[sure]).all()


_ATTENTION = [pytest.param(*c[1:], D, cache, id=f"{c[0][0]}rows-{c[0][1 + (cache == 'e4m3')]}groups-"
                           f"{'split' if c[0][3] else 'whole'}-{D}-{cache}")
              for c in lc.ATTENTION_SINKS for D in (64, 128) for cache in ("bf16", "e4m3")]


@pytest.mark.parametrize("ctx,chunk,Hq,Hk,P,window,sinks,more,D,cache", _ATTENTION)
def test_attention(ctx, chunk, Hq, Hk, P, window, sinks, more, D, cache):
    # against float64, with NaN in every page and behind every end that no row sees
    _case(ctx, chunk, Hq, Hk, D, P, window, sinks, cache=cache, seed=Hq + D, **more)


@pytest.mark.parametrize("ctx,chunk,Hq,Hk,P,window,sinks,more,D,cache", _ATTENTION)
def test_attention_with_values_that_are_no_numbers(ctx, chunk, Hq, Hk, P, window, sinks, more, D, cache):
    # of the first key, which all see, of the key in the middle of a request's new tokens, and of one that the window of only
    # some of its tokens reaches: each reaches the rows that see it, in its own column, and no others
    import torch
    import markov_draft_sampling_amd as mds
    causal = more.get("causal", True)
    g = torch.Generator().manual_seed(Hq)
    seq = [a + n for a, n in zip(ctx, chunk)]
    MP = -(-max(seq) // P)
    used = sum(-(-x // P) for x in seq)
    kind = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
    kp, vp = (torch.randn((used, P, Hk, D), generator=g).to(kind) for _ in range(2))
    raw = vp.view(torch.uint8 if cache == "e4m3" else torch.int16)
    nan, inf = (0x7F, 0x7F) if cache == "e4m3" else (0x7FC0, 0x7F80)  # (e4m3 has no infinities)
    table = torch.full((len(ctx), MP), -1, dtype=torch.int32)
    expect = torch.zeros((sum(chunk), 3), dtype=torch.bool)
    at = t0 = 0
    for b, (c, n) in enumerate(zip(ctx, chunk)):
        held = -(-seq[b] // P)
        table[b, :held] = torch.arange(at, at + held, dtype=torch.int32)
        pos = torch.arange(c, c + n)
        for i, key in enumerate((0, c + n // 2, max(0, c - window + 1 + n // 2)) if n else ()):
            seen = (key <= pos) if causal else torch.ones(n, dtype=torch.bool)
            expect[t0:t0 + n, i] = seen & ((key > pos - window) | (key < sinks))
            raw[at + key // P, key % P, :, 5 + 20 * i] = inf if i == 1 else nan
        at, t0 = at + held, t0 + n
    T = sum(chunk)
    q = torch.randn((T, Hq, D), generator=g).to(torch.bfloat16).cuda()
    out = torch.zeros_like(q)
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    starts = t(np.concatenate([[0], np.cumsum(chunk)]).tolist())
    ws = mds.paged_attention(q, kp.cuda(), vp.cuda(), table.cuda(), starts, t(seq), out, max(chunk), max(seq), window=window,
                             sinks=sinks, causal=causal)
    assert mds.workspace_status(ws) == 0
    o = out.float().cpu()
    for i in range(3):
        x, hit = o[:, :, 5 + 20 * i], expect[:, i]
        assert (x[hit] == math.inf if i == 1 and cache == "bf16" else x[hit].isnan()).all(), i
        assert x[~hit].isfinite().all(), i
    rest = [d for d in range(D) if d not in (5, 25, 45)]
    assert o[:, :, rest].isfinite().all()
