"""Norm and rotation on the GPU against float64 within the bounds of their
float32 arithmetic: both layouts, part of a head, far positions, strides,
outputs over inputs, padding; and the append in the same pass against the two
calls it stands for."""
from __future__ import annotations

import numpy as np
import pytest

import layer_ref as lr
import serving_ref as sr

pytestmark = pytest.mark.gpu


def _inputs(T, Hq, Hk, D, R, norm=True, seed=0, far=100000, layout="qkv"):
    import torch
    import markov_draft_sampling_amd as mds
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, Hq + 2 * Hk, D), generator=g) * (0.1 + 4 * torch.rand((1, Hq + 2 * Hk, 1), generator=g))
    if T:
        x[0, 0] = 0  # a head of zeros
    d = x.to(torch.bfloat16).cuda()
    if layout == "htd":
        d = d.transpose(0, 1).contiguous().transpose(0, 1)
    elif layout == "padded":
        wide = torch.full((T, Hq + 2 * Hk, D + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[..., :D] = d
        d = wide[..., :D]
    s = dict(q=d[:, :Hq], k=d[:, Hq:Hq + Hk], v=d[:, Hq + Hk:], qw=None, kw=None)
    if norm:
        for n in ("qw", "kw"):
            s[n] = (1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda()
    s["pos"] = torch.randint(0, far, (T,), generator=g).cuda()
    if T > 2:
        s["pos"][1], s["pos"][2] = 0, far
    s["freq"] = mds.rope_frequencies(R)[0] if R else None
    return s


def _expected(s, rope_scale=1.0, interleaved=False, eps=1e-6):
    c = lambda t: None if t is None else t.cpu()  # noqa: E731
    return [lr.norm_rope(s[n].cpu(), c(s[w]), eps, s["pos"].cpu(), c(s["freq"]), interleaved, rope_scale)
            for n, w in (("q", "qw"), ("k", "kw"))]


def _check(got, ref, err):
    # rounded once to bf16: half a step is 2^-8 of the value
    e = (got.cpu().double() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() + 1.01 * err + 1e-37
    assert (e <= tol).all(), float((e / tol).max())


def _run(T, Hq, Hk, D, R, interleaved=False, norm=True, rope_scale=1.0, eps=1e-6, seed=0, far=100000, layout="qkv"):
    import torch
    import markov_draft_sampling_amd as mds
    s = _inputs(T, Hq, Hk, D, R, norm, seed, far, layout)
    print(f"rope T {T} heads {Hq}/{Hk} D {D} R {R} interleaved {interleaved} norm {norm} {layout}", flush=True)
    pad = 2
    qo = torch.full((T + pad, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((T + pad, Hk, D), 7.0, dtype=torch.bfloat16, device="cuda")
    args = dict(q_weight=s["qw"], k_weight=s["kw"], eps=eps, interleaved=interleaved, rope_scale=rope_scale)
    mds.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], qo[:T], ko[:T], **args)
    torch.cuda.synchronize()
    (q, eq), (k, ek) = _expected(s, rope_scale, interleaved, eps)
    _check(qo[:T], q, eq)
    _check(ko[:T], k, ek)
    assert (qo[T:] == 7).all() and (ko[T:] == 7).all()
    again = qo.clone()
    mds.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], qo[:T], ko[:T], **args)
    assert torch.equal(again, qo)
    # over its own input
    mds.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], s["q"], s["k"], **args)
    assert torch.equal(s["q"], qo[:T]) and torch.equal(s["k"], ko[:T])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 32), (128, 128), (128, 16), (80, 80), (96, 48), (192, 96), (256, 256),
                                 (16, 16), (112, 0)])
def test_norm_and_rotation(D, R, norm, interleaved):
    _run(5, 6, 2, D, R, interleaved, norm)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 32, 8), (3, 5, 1), (7, 8, 8), (33, 3, 2), (300, 32, 8), (2, 130, 66),
                                     (1025, 7, 3)])
def test_tokens_and_heads(T, Hq, Hk):
    _run(T, Hq, Hk, 128, 128, seed=T)
    _run(T, Hq, Hk, 64, 32, interleaved=True, seed=T)


@pytest.mark.parametrize("layout", ["htd", "padded"])
def test_strides(layout):
    _run(9, 6, 2, 128, 64, layout=layout)
    _run(9, 6, 2, 64, 64, interleaved=True, layout=layout)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 1, 1 << 40])
def test_far_positions(far):
    _run(40, 2, 1, 128, 128, far=far, rope_scale=1.37, eps=1e-5)
    _run(40, 2, 1, 64, 64, far=far, interleaved=True, norm=False)


def test_one_of_the_two_norms():
    import torch
    import markov_draft_sampling_amd as mds
    s = _inputs(6, 4, 2, 128, 128)
    for drop in ("qw", "kw"):
        t = {**s, drop: None}
        qo, ko = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
        mds.qk_norm_rope(t["q"], t["k"], t["pos"], t["freq"], qo, ko, q_weight=t["qw"], k_weight=t["kw"])
        (q, eq), (k, ek) = _expected(t)
        _check(qo, q, eq)
        _check(ko, k, ek)


def test_infinities_and_nan_stay_in_their_heads():
    import torch
    import markov_draft_sampling_amd as mds
    s = _inputs(4, 9, 3, 128, 64)
    clean_q, clean_k = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
    run = lambda q, k: mds.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], q, k, q_weight=s["qw"],  # noqa: E731
                                        k_weight=s["kw"])
    run(clean_q, clean_k)
    s["q"][1, 3, 5] = float("nan")
    s["k"][2, 1, 100] = float("nan")
    qo, ko = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
    run(qo, ko)
    bad_q, bad_k = torch.zeros(4, 9, dtype=torch.bool), torch.zeros(4, 3, dtype=torch.bool)
    bad_q[1, 3], bad_k[2, 1] = True, True
    assert qo[1, 3].isnan().all() and ko[2, 1].isnan().all()  # the sum of squares has it
    assert torch.equal(qo.cpu()[~bad_q], clean_q.cpu()[~bad_q]) and torch.equal(ko.cpu()[~bad_k], clean_k.cpu()[~bad_k])


def _pages(NP, P, H, D, cache, layout, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((NP, P, H, D), generator=g).to(torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn).cuda()
    if layout == "hnd":
        b = x.view(torch.uint8 if cache == "e4m3" else x.dtype)
        x = b.transpose(1, 2).contiguous().transpose(1, 2).view(x.dtype)
    return x


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,Hq,Hk,D,R,interleaved,norm,P,layout", [
    (1, 32, 8, 128, 128, False, True, 16, "nhd"), (37, 6, 2, 64, 64, False, True, 16, "hnd"),
    (37, 5, 3, 128, 64, True, False, 32, "nhd"), (130, 4, 4, 80, 48, True, True, 64, "hnd"),
    (65, 3, 1, 256, 128, False, True, 16, "nhd"), (9, 70, 2, 192, 16, False, False, 128, "nhd")])
def test_the_append_in_the_same_pass(T, Hq, Hk, D, R, interleaved, norm, P, layout, cache):
    import torch
    import markov_draft_sampling_amd as mds
    s = _inputs(T, Hq, Hk, D, R, norm, seed=T)
    rng = np.random.default_rng(T)
    NP = -(-T // P) + 3
    slot = rng.permutation(NP * P)[:T].astype(np.int64)
    if T > 3:
        slot[1] = -1
        slot[T - 1] = -5
    ks = vs = None
    if cache == "e4m3":
        ks, vs = (torch.tensor(rng.uniform(0.002, 0.03, Hk), dtype=torch.float32).cuda() for _ in range(2))
    kp, vp = _pages(NP, P, Hk, D, cache, layout, 1), _pages(NP, P, Hk, D, cache, layout, 2)
    before = [x.float().cpu().view(NP * P, Hk, D) if layout == "nhd" else x.float().cpu().reshape(NP * P, Hk, D)
              for x in (kp, vp)]
    want_k, want_v = kp.clone(), vp.clone()
    sl = torch.from_numpy(slot).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    args = dict(q_weight=s["qw"], k_weight=s["kw"], interleaved=interleaved, rope_scale=1.1)
    print(f"rope append T {T} heads {Hq}/{Hk} D {D} R {R} {cache} {layout}", flush=True)
    mds.qk_norm_rope_append(s["q"], s["k"], s["v"], s["pos"], s["freq"], qo, kp, vp, sl, k_scale=ks, v_scale=vs,
                            status=status, **args)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    q2, k2 = torch.zeros_like(qo), torch.zeros((T, Hk, D), dtype=torch.bfloat16, device="cuda")
    mds.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], q2, k2, **args)
    assert torch.equal(qo, q2)  # padding rows too
    mds.kv_append(k2, s["v"], want_k, want_v, sl, k_scale=ks, v_scale=vs)
    bits = lambda t: t.view(torch.uint8 if cache == "e4m3" else torch.int16).cpu()  # noqa: E731
    assert torch.equal(bits(vp), bits(want_v))
    if cache == "bf16":
        assert torch.equal(bits(kp), bits(want_k))
        return
    # 8-bit keys, rounded once: half a step (2^-4, or 2^-10 below the normal codes), on what float32 leaves of y / scale
    _, (ref, err) = _expected(s, 1.1, interleaved)
    live = slot >= 0
    got = kp.float().cpu().reshape(NP * P, Hk, D)
    sc = ks.cpu().double()[:, None]
    z = (ref / sc).clamp(-448, 448)[torch.from_numpy(live)]
    e = (got[slot[live]].double() - z).abs()
    fuzz = (err / sc + 2.0 ** -23 * (ref / sc).abs())[torch.from_numpy(live)] * 1.01
    # where the quotient is near the border between two codes either may come: half a step of the larger one
    tol = torch.maximum(2.0 ** -4 * (z.abs() + fuzz), torch.tensor(2.0 ** -10)) + fuzz
    assert (e <= tol).all(), float((e / tol).max())
    # and the code is the nearest one wherever float32 cannot tell them apart
    near = sr.e4m3_round(z.float().numpy())
    lo, hi = sr.e4m3_round((z - fuzz).float().numpy()), sr.e4m3_round((z + fuzz).float().numpy())
    sure = lo == hi
    assert sure.mean() > 0.99 and (got[slot[live]].double().numpy()[sure] == near[sure]).all()
    rest = np.setdiff1d(np.arange(NP * P), slot[live])
    assert torch.equal(got[rest], before[0][rest])


@pytest.mark.parametrize("D,interleaved,norm", [(64, False, True), (128, False, True), (128, True, True), (256, True, True),
                                                (96, False, False), (128, True, False)])
def test_codes_are_those_of_separate_operations(D, interleaved, norm):
    # The float32 factors nearest to their exact values, each operation rounded by itself, squares in the columns' order:
    # the codes are equal but where a float64 sine or root lies within 2^-50 of the middle of two float32s (one in 10^4
    # sines at these positions) and the code within 2^-23 of the border of two (one in 10^6): 10^-5 in all for 10^5 keys.
    import torch
    import markov_draft_sampling_amd as mds
    T, Hk = 96, 8
    s = _inputs(T, 4, Hk, D, D, norm, seed=D)
    scale = torch.linspace(0.003, 0.03, Hk)
    kp, vp = (torch.zeros((T // 16, 16, Hk, D), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    mds.qk_norm_rope_append(s["q"], s["k"], s["v"], s["pos"], s["freq"], torch.empty_like(s["q"]), kp, vp,
                            torch.arange(T).cuda(), q_weight=s["qw"], k_weight=s["kw"], interleaved=interleaved,
                            rope_scale=1.2079441541679836, k_scale=scale.cuda(), v_scale=scale.cuda())
    k = s["k"].cpu().float()
    if norm:
        z = (k * k).view(T, Hk, D // 4, 4)
        z = ((z[..., 0] + z[..., 1]) + z[..., 2]) + z[..., 3]
        while z.shape[-1] > 1:
            z = z[..., 0::2] + z[..., 1::2]
        k = k * (z / D + 1e-6).double().rsqrt().float() * s["kw"].cpu().float()
    a = s["pos"].cpu().double()[:, None] * s["freq"].cpu()
    c, n = ((f(a) * 1.2079441541679836).float()[:, None] for f in (torch.cos, torch.sin))
    p, q = (k[..., 0::2], k[..., 1::2]) if interleaved else (k[..., :D // 2], k[..., D // 2:])
    y, z = p * c - q * n, q * c + p * n
    k = torch.stack([y, z], -1).flatten(-2) if interleaved else torch.cat([y, z], -1)
    for got, x in ((kp, k), (vp, s["v"].cpu().float())):
        want = (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(got.view(torch.uint8).cpu().view(T, Hk, D), want.view(torch.uint8))


def test_slots_past_the_cache_are_flagged_and_skipped():
    import torch
    import markov_draft_sampling_amd as mds
    s = _inputs(5, 4, 2, 64, 64, norm=False)
    kp, vp = _pages(2, 16, 2, 64, "bf16", "nhd", 1), _pages(2, 16, 2, 64, "bf16", "nhd", 2)
    k0, v0 = kp.clone(), vp.clone()
    slot = torch.tensor([3, 32, -1, 1 << 40, 31], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = torch.zeros_like(s["q"])
    mds.qk_norm_rope_append(s["q"], s["k"], s["v"], s["pos"], s["freq"], qo, kp, vp, slot, status=status)
    assert int(status.item()) == mds.STATUS_BAD_PAGE
    changed = ((kp != k0).flatten(2).any(-1) | (vp != v0).flatten(2).any(-1)).view(-1).nonzero().view(-1).tolist()
    assert changed == [3, 31]
    (q, eq), _ = _expected(s)
    _check(qo, q, eq)


def test_other_streams_and_a_graph():
    import torch
    import markov_draft_sampling_amd as mds
    s = _inputs(64, 8, 2, 128, 128)
    kp, vp = _pages(8, 16, 2, 128, "bf16", "nhd", 1), _pages(8, 16, 2, 128, "bf16", "nhd", 2)
    slot = torch.randperm(128)[:64].cuda()
    qo, want = torch.zeros_like(s["q"]), torch.zeros_like(s["q"])
    kw, vw = kp.clone(), vp.clone()
    args = dict(q_weight=s["qw"], k_weight=s["kw"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mds.qk_norm_rope_append(s["q"], s["k"], s["v"], s["pos"], s["freq"], qo, kp, vp, slot, stream=side, **args)
    side.synchronize()
    mds.qk_norm_rope_append(s["q"], s["k"], s["v"], s["pos"], s["freq"], want, kw, vw, slot, **args)
    assert torch.equal(qo, want) and torch.equal(kp, kw) and torch.equal(vp, vw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mds.qk_norm_rope_append(s["q"], s["k"], s["v"], s["pos"], s["freq"], qo, kp, vp, slot, **args)
    for i in range(4):
        s["pos"].add_(17)
        s["q"].mul_(1.5)
        slot.copy_(torch.randperm(128)[:64])
        g.replay()
        mds.qk_norm_rope_append(s["q"], s["k"], s["v"], s["pos"], s["freq"], want, kw, vw, slot, **args)
        torch.cuda.synchronize()
        assert torch.equal(qo, want) and torch.equal(kp, kw) and torch.equal(vp, vw), i


def test_refusals_of_the_binding():
    import torch
    import markov_draft_sampling_amd as mds
    s = _inputs(4, 4, 2, 64, 64)
    qo, ko = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
    ok = dict(q=s["q"], k=s["k"], positions=s["pos"], inv_freq=s["freq"], q_out=qo, k_out=ko)
    mds.qk_norm_rope(**ok)
    for bad in (dict(q=s["q"].float()), dict(k=s["k"][:3]), dict(positions=s["pos"].int()), dict(positions=s["pos"][:3]),
                dict(inv_freq=s["freq"].float()), dict(q_out=qo[:, :3]), dict(k_out=ko.float()), dict(k_out=ko.cpu()),
                dict(q_weight=torch.ones(64, device="cuda")), dict(k_weight=torch.ones(32, dtype=torch.bfloat16).cuda()),
                dict(q=s["q"][..., ::2]), dict(eps=-1.0), dict(inv_freq=s["freq"][:4]),
                dict(q_out=torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda").expand(4, 4, 64))):
        with pytest.raises(mds.MdsError):
            mds.qk_norm_rope(**{**ok, **bad})
    kp, vp = _pages(2, 16, 2, 64, "bf16", "nhd", 1), _pages(2, 16, 2, 64, "bf16", "nhd", 2)
    slot = torch.arange(4, device="cuda")
    ok = dict(q=s["q"], k=s["k"], v=s["v"], positions=s["pos"], inv_freq=s["freq"], q_out=qo, k_pages=kp, v_pages=vp,
              slot_map=slot)
    mds.qk_norm_rope_append(**ok)
    for bad in (dict(v=s["v"][:, :1]), dict(slot_map=slot.int()), dict(slot_map=slot[:3]), dict(k_pages=kp[:, :, :1]),
                dict(k_pages=kp[..., :32], v_pages=vp[..., :32]), dict(v_pages=vp.float()),
                dict(k_pages=kp.to(torch.float8_e4m3fn), v_pages=vp.to(torch.float8_e4m3fn)),
                dict(status=torch.zeros(2, device="cuda"))):
        with pytest.raises(mds.MdsError):
            mds.qk_norm_rope_append(**{**ok, **bad})


def test_threads_of_the_interpreter():
    # the calls let other threads run while they enqueue; errors belong to the thread whose call it was
    import threading
    import torch
    import markov_draft_sampling_amd as mds
    sets = [_inputs(32 + 8 * i, 8, 2, 128, 128, seed=i) for i in range(4)]
    want = []
    for s in sets:
        q, k = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        mds.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], q, k, q_weight=s["qw"], k_weight=s["kw"])
        want.append((q, k))
    torch.cuda.synchronize()
    failed = []

    def work(i):
        s, st = sets[i], torch.cuda.Stream()
        q, k = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        try:
            for n in range(100):
                args = dict(q_weight=s["qw"], k_weight=s["kw"], stream=st)
                if n % 10 == i:
                    with pytest.raises(mds.MdsError, match="eps" if i % 2 else "rope_scale"):
                        mds.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], q, k, eps=-1.0 if i % 2 else 1e-6,
                                         rope_scale=1.0 if i % 2 else float("nan"), **args)
                mds.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], q, k, **args)
            st.synchronize()
            assert torch.equal(q, want[i][0]) and torch.equal(k, want[i][1])
        except BaseException as e:  # noqa: BLE001
            failed.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
