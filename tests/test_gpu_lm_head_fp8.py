"""The 8-bit LM head on the GPU against float64 within the bound of its float32
sums: products of codes are exact; a block's sum of 128 products is float32
(2^-23 a term for a sum that truncates), scaled (three roundings) and added
to the total of H / 128 blocks; then the output's own rounding."""
from __future__ import annotations

import numpy as np
import pytest

import serving_ref as sr
import workloads

pytestmark = pytest.mark.gpu


def _weights(V, H, seed, mode):
    """(e4m3 values float64 [V, H], scales, tiled device tensor, scales device tensor)."""
    import torch
    import markov_draft_sampling_amd as mds
    rng = np.random.default_rng(seed)
    w = (rng.standard_normal((V, H)) * 3 / np.sqrt(H)).astype(np.float32)
    w[:: max(1, V // 7), : 128] = 0  # rows and a block of zeros
    if V > 130:
        w[128:256, :128] = 0
    bits = torch.from_numpy(w).to(torch.bfloat16)
    w = bits.float().numpy()
    q, s = sr.quantize_blocks(w, 128, 128)
    if mode == "quantize":
        tiled, sd = mds.quantize_lm_head_fp8(bits.cuda())
        assert np.array_equal(sd.cpu().numpy(), s)
    else:
        codes = torch.from_numpy(q.astype(np.float32)).to(torch.float8_e4m3fn).cuda()
        tiled, sd = mds.tile_lm_head_fp8(codes), torch.from_numpy(s).cuda()
    return q, s, tiled, sd


def _run(B, K, V, H, seed=0, out_dtype="f32", mode="quantize", pad=0, extra=0):
    import torch
    import markov_draft_sampling_amd as mds
    rng = np.random.default_rng(seed + 100)
    q, s, tiled, sd = _weights(V, H, seed, mode)
    x = rng.standard_normal((B * K, H)).astype(np.float32)
    x[:, rng.integers(0, H, 3)] *= 20
    x[0, :128] = 0
    xb = torch.zeros((B * K, H + 8), dtype=torch.bfloat16)
    xb[:, :H] = torch.from_numpy(x)
    hidden = xb.cuda()[:, :H]
    xq, xs = sr.quantize_blocks(xb[:, :H].float().numpy(), 1, 128)
    dt = torch.bfloat16 if out_dtype == "bf16" else torch.float32
    out = torch.full((B, K + extra, V + pad), 7.25, dtype=dt, device="cuda")
    print(f"8-bit LM head B {B} K {K} V {V} H {H} {out_dtype} {mode}", flush=True)
    mds.lm_head_fp8(hidden, tiled, sd, out[..., :V], K)
    torch.cuda.synchronize()
    o = out.float().cpu().numpy()
    assert (o[:, K:] == 7.25).all() and (o[..., V:] == 7.25).all()
    got = o[:, :K, :V].reshape(B * K, V).astype(np.float64)
    z, a = sr.lm_head(xq, xs, q, s)
    tol = (2 * 128 + H // 128 + 4) * 2.0 ** -24 * a + 2.0 ** -24 * np.abs(z)
    if out_dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(z)
    err = np.abs(got - z)
    assert (err <= tol).all(), (np.argwhere(err > tol)[:4], float((err / np.maximum(tol, 1e-30)).max()))


@pytest.mark.parametrize("B,K,V,H", [(1, 1, 2, 128), (1, 7, 4099, 256), (3, 5, 130, 384), (8, 4, 999, 1024),
                                     (9, 7, 1000, 640), (20, 7, 2050, 256), (27, 7, 515, 512), (32, 7, 3001, 256),
                                     (33, 7, 700, 256), (64, 8, 300, 128)])
@pytest.mark.parametrize("mode", ["quantize", "tile"])
def test_lm_head_fp8(B, K, V, H, mode):
    _run(B, K, V, H, seed=B + V, mode=mode)


@pytest.mark.parametrize("rows", [17, 32, 33, 48, 64, 66, 84, 112, 126, 140, 170, 224])
@pytest.mark.parametrize("V", [20003, 33003, 65701])
def test_every_row_tile_and_vocabulary_width(rows, V):
    _run(rows, 1, V, 128, seed=rows)


@pytest.mark.parametrize("rows", [1, 7, 16, 17, 32])
@pytest.mark.parametrize("H", [128, 256, 384, 512, 640, 768, 896, 1664])
def test_few_rows_over_every_fill_of_the_ring(rows, H):
    # fewer chunks of 128 columns than the ring has places, as many, and more, once and twice around
    _run(1 if rows <= 16 else rows, rows if rows <= 16 else 1, 1021, H, seed=rows + H)


@pytest.mark.parametrize("H", [384, 640, 1024])
@pytest.mark.parametrize("V", [33003, 65701])
def test_wide_vocabularies_over_several_chunks(V, H):
    # work-groups of two and of four vocabulary blocks a wave, over an odd and an even number of chunks of 128 columns;
    # checked at the first, the last and some other vocabulary rows
    import torch
    import markov_draft_sampling_amd as mds
    g = torch.Generator().manual_seed(V + H)
    codes = torch.randint(0, 127, (V, H), generator=g, dtype=torch.uint8)  # 127 is NaN
    codes |= torch.randint(0, 2, (V, H), generator=g, dtype=torch.uint8) << 7
    codes = codes.view(torch.float8_e4m3fn)
    scales = torch.rand(((V + 127) // 128, H // 128), generator=g) * 1e-3 + 1e-4
    tiled, sd = mds.tile_lm_head_fp8(codes.cuda()), scales.cuda()
    at = np.unique(np.concatenate([np.arange(140), np.arange(V - 140, V), np.random.default_rng(V).integers(0, V, 400)]))
    wq = codes[torch.from_numpy(at)].float().numpy().astype(np.float64)
    ws = scales.numpy()[at // 128]
    x = torch.randn((224, H), generator=g).to(torch.bfloat16)
    xq, xs = sr.quantize_blocks(x.float().numpy(), 1, 128)
    z = a = 0
    for j in range(H // 128):
        c = slice(j * 128, (j + 1) * 128)
        xj, wj = xq[:, c] * xs[:, j:j + 1].astype(np.float64), wq[:, c] * ws[:, j:j + 1].astype(np.float64)
        z, a = z + xj @ wj.T, a + np.abs(xj) @ np.abs(wj).T
    tol = (2 * 128 + H // 128 + 4) * 2.0 ** -24 * a + 2.0 ** -24 * np.abs(z)
    for rows in (32, 33, 64, 112, 126, 224):
        print(f"8-bit LM head rows {rows} V {V} H {H}", flush=True)
        out = torch.full((rows, 1, V), 7.25, device="cuda")
        mds.lm_head_fp8(x[:rows].cuda(), tiled, sd, out, 1)
        got = out[:, 0].cpu().numpy()[:, at].astype(np.float64)
        err = np.abs(got - z[:rows])
        assert (err <= tol[:rows]).all(), (rows, np.argwhere(err > tol[:rows])[:4])


def test_lm_head_fp8_bf16_out_strided_with_rows_left_alone():
    _run(6, 8, 1003, 256, seed=1, out_dtype="bf16", pad=5, extra=2)
    _run(6, 8, 1003, 256, seed=1, out_dtype="f32", pad=5, extra=2)
    _run(6, 8, 1004, 256, seed=2, out_dtype="bf16", pad=4)


def test_tiled_order_and_quantised_codes():
    import torch
    V, H = 300, 256
    q, s, tiled, sd = _weights(V, H, 3, "quantize")
    t = tiled.float().cpu().numpy().reshape(-1)
    v, c = np.meshgrid(np.arange(V), np.arange(H), indexing="ij")
    at = ((v // 16) * (H // 128) + c // 128) * 2048 + ((c % 128) // 16) * 256 + (v % 16) * 16 + c % 16
    assert np.array_equal(t[at], q)
    rest = np.ones(t.size, bool)
    rest[at] = False
    assert (t[rest] == 0).all()
    _, _, tiled2, _ = _weights(V, H, 3, "tile")
    # (a zero's sign aside)
    assert torch.equal(tiled.float(), tiled2.float())


def test_rows_with_nan_or_infinity_are_nan_and_leave_the_others():
    import torch
    import markov_draft_sampling_amd as mds
    V, H = 200, 256
    _, _, tiled, sd = _weights(V, H, 4, "quantize")
    x = torch.randn(6, H, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    clean = torch.empty((6, 1, V), device="cuda")
    mds.lm_head_fp8(x.cuda(), tiled, sd, clean, 1)
    x[1, 5], x[3, 200], x[4, 130] = float("nan"), float("inf"), -float("inf")
    out = torch.empty((6, 1, V), device="cuda")
    mds.lm_head_fp8(x.cuda(), tiled, sd, out, 1)
    assert torch.isnan(out[[1, 3, 4]]).all()
    assert torch.equal(out[[0, 2, 5]], clean[[0, 2, 5]])


def test_lm_head_fp8_feeds_the_draft_loop():
    """The 8-bit head's base logits drive the loop: tokens as from the same logits in a buffer."""
    import torch
    import markov_draft_sampling_amd as mds
    wl = workloads.make_custom(4096, 64, 3, 4, seed=6)
    _, _, tiled, sd = _weights(wl.V, 256, 6, "quantize")
    hidden = torch.randn(wl.B * wl.K, 256, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    base = torch.zeros((wl.B, wl.K + 1, wl.V), dtype=torch.float32, device="cuda")
    mds.lm_head_fp8(hidden, tiled, sd, base, wl.K)
    import oracle
    w1 = torch.from_numpy(wl.w1.view(np.int16)).view(torch.bfloat16).cuda()
    w2 = torch.from_numpy(wl.w2.view(np.int16)).view(torch.bfloat16).cuda()
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    cache = torch.empty((wl.B, wl.K, wl.V), dtype=torch.float32, device="cuda")
    toks = torch.empty((wl.B, wl.K), dtype=torch.int32, device="cuda")
    mds.markov_draft_loop(base, w1, w2, t(wl.anchor_tokens), t(wl.anchor_pos), t(wl.temperature), t(wl.seeds), cache,
                          toks)
    g = toks.cpu().numpy()
    ref = oracle.draft_loop(base.cpu().numpy(), "f32", wl.w1, wl.w2, wl.anchor_tokens, wl.anchor_pos, wl.seeds,
                            wl.temperature, "f32", K=wl.K, teacher=g)
    assert not ((ref["tokens"] != g) & (ref["margin"] > 1e-3)).any()


def test_lm_head_fp8_graph_replays():
    import torch
    import markov_draft_sampling_amd as mds
    V, H = 3000, 512
    _, _, tiled, sd = _weights(V, H, 8, "quantize")
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(14, H, generator=gen).to(torch.bfloat16).cuda()
    out = torch.empty((2, 7, V), device="cuda")
    ws = mds.new_workspace(mds.lm_head_fp8_workspace_bytes(2, 7, V, H))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mds.lm_head_fp8(x, tiled, sd, out, 7, workspace=ws)
    for _ in range(4):
        x.copy_(torch.randn(14, H, generator=gen).to(torch.bfloat16).cuda())
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(out)
        mds.lm_head_fp8(x, tiled, sd, want, 7)
        assert torch.equal(out, want)


def test_side_stream_makes_its_outputs_there():
    import torch
    import markov_draft_sampling_amd as mds
    V, H = 3000, 512
    w, _, tiled, sd = _weights(V, H, 8, "quantize")
    wd = torch.randn(V, H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    want, want_s = mds.quantize_lm_head_fp8(wd)
    codes = torch.randint(0, 120, (V, H), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    want_t = mds.tile_lm_head_fp8(codes)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    # memory that the current stream still writes, freed for whoever asks on that stream
    busy = torch.zeros(V * H, dtype=torch.uint8, device="cuda")
    for i in range(20):
        busy.add_(1)
    del busy
    got, got_s = mds.quantize_lm_head_fp8(wd, stream=side)
    got_t = mds.tile_lm_head_fp8(codes, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    u8 = lambda x: x.view(torch.uint8)  # noqa: E731
    assert torch.equal(u8(got), u8(want)) and torch.equal(got_s, want_s) and torch.equal(u8(got_t), u8(want_t))


def test_one_row_of_any_stride():
    import torch
    import markov_draft_sampling_amd as mds
    V, H = 1000, 256
    _, _, tiled, sd = _weights(V, H, 3, "quantize")
    x = torch.randn(1, H, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    out, out2 = torch.empty(1, 1, V, device="cuda"), torch.empty(1, 1, V, device="cuda")
    mds.lm_head_fp8(x, tiled, sd, out, 1)
    mds.lm_head_fp8(x.as_strided((1, H), (0, 1)), tiled, sd, out2.as_strided((1, 1, V), (3, 1, 1)), 1)
    assert torch.equal(out, out2)


def test_refuses_mismatched_tensors():
    import torch
    import markov_draft_sampling_amd as mds
    _, _, tiled, sd = _weights(200, 256, 4, "quantize")
    x = torch.zeros(6, 256, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(2, 3, 200, device="cuda")
    mds.lm_head_fp8(x, tiled, sd, out, 3)
    for bad in (dict(x=x.float()), dict(x=x[:5]), dict(t=tiled[:-1]), dict(s=sd[:1]), dict(o=out.half()),
                dict(o=out[:, :2]), dict(o=out.cpu()), dict(t=tiled.cpu())):
        a = dict(x=x, t=tiled, s=sd, o=out)
        a.update(bad)
        with pytest.raises(mds.MdsError):
            mds.lm_head_fp8(a["x"], a["t"], a["s"], a["o"], 3)
    with pytest.raises(mds.MdsError):
        mds.quantize_lm_head_fp8(torch.zeros(100, 100, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(mds.MdsError):
        mds.tile_lm_head_fp8(torch.zeros(100, 256, dtype=torch.bfloat16, device="cuda"))
