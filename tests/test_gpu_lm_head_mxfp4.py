"""The 4-bit LM head on the GPU against float64: codes, scales and their
order exactly; logits within the bound of their float32 sums: products are
exact, a matrix instruction adds 32 of them to a sum with at most two
roundings (or truncations: 2^-23) of a partial sum that sum |x w| = A bounds,
H / 32 instructions follow each other, and four sums are joined."""
from __future__ import annotations

import numpy as np
import pytest

import layer_ref as lr

pytestmark = pytest.mark.gpu


def _matrix(V, H, seed, mode):
    """(weights float64 [V, H], tiled codes, tiled scales on the device)."""
    import torch
    import markov_draft_sampling_amd as mds
    rng = np.random.default_rng(seed)
    if mode == "quantize":
        w = (rng.standard_normal((V, H)) * 3 / np.sqrt(H) * rng.uniform(0.1, 2, (V, 1))).astype(np.float32)
        w[:: max(1, V // 7), :64] = 0
        bits = torch.from_numpy(w).to(torch.bfloat16)
        codes, scales = lr.mx_quantize(bits.float().numpy())
        tiled, ts = mds.quantize_lm_head_mxfp4(bits.cuda())
    else:
        codes = rng.integers(0, 16, (V, H)).astype(np.uint8)
        scales = rng.integers(117, 124, (V, H // 32)).astype(np.uint8)
        tiled, ts = mds.tile_lm_head_mxfp4(torch.from_numpy(lr.mx_pack(codes)).cuda(), torch.from_numpy(scales).cuda())
    return lr.mx_values(codes, scales), codes, scales, tiled, ts


def _check(got, x, w, bf16=False):
    H = x.shape[1]
    z, a = x @ w.T, np.abs(x) @ np.abs(w).T
    tol = (4 * H / 32 + 16) * 2.0 ** -24 * a + 1e-37
    if bf16:
        tol = tol + 2.0 ** -8 * (np.abs(z) + tol)
    err = np.abs(got - z)
    assert (err <= tol).all(), (np.argwhere(~(err <= tol))[:4], float((err / tol).max()))


def _run(B, K, V, H, seed=0, out_dtype="f32", mode="tile", pad=0, extra=0):
    import torch
    import markov_draft_sampling_amd as mds
    w, _, _, tiled, ts = _matrix(V, H, seed, mode)
    rng = np.random.default_rng(seed + 100)
    x = rng.standard_normal((B * K, H)).astype(np.float32)
    x[:, rng.integers(0, H, 3)] *= 20
    xb = torch.full((B * K, H + 8), float("nan"), dtype=torch.bfloat16)
    xb[:, :H] = torch.from_numpy(x)
    out = torch.full((B, K + extra, V + pad), 7.25, dtype=torch.bfloat16 if out_dtype == "bf16" else torch.float32,
                     device="cuda")
    print(f"4-bit LM head B {B} K {K} V {V} H {H} {out_dtype} {mode}", flush=True)
    hidden = xb.cuda()[:, :H]
    mds.lm_head_mxfp4(hidden, tiled, ts, out[..., :V], K)
    torch.cuda.synchronize()
    o = out.float().cpu().numpy()
    assert (o[:, K:] == 7.25).all() and (o[..., V:] == 7.25).all()
    _check(o[:, :K, :V].reshape(B * K, V).astype(np.float64), xb[:, :H].double().numpy(), w, out_dtype == "bf16")
    again = out.clone()
    mds.lm_head_mxfp4(hidden, tiled, ts, out[..., :V], K)
    assert torch.equal(again, out)


@pytest.mark.parametrize("B,K,V,H", [(1, 1, 2, 128), (1, 7, 4099, 256), (3, 5, 130, 384), (8, 4, 999, 1024),
                                     (9, 7, 1000, 640), (20, 7, 2050, 256), (27, 7, 515, 512), (32, 7, 3001, 256),
                                     (33, 7, 700, 256), (64, 8, 300, 128), (2, 8, 17, 4096)])
@pytest.mark.parametrize("mode", ["quantize", "tile"])
def test_lm_head_mxfp4(B, K, V, H, mode):
    _run(B, K, V, H, seed=B + V, mode=mode)


@pytest.mark.parametrize("rows", [1, 16, 17, 32, 33, 48, 64, 66, 84, 96, 112, 126, 140, 170, 224, 240])
@pytest.mark.parametrize("V", [5003, 33003])
def test_every_row_tile(rows, V):
    _run(rows, 1, V, 128, seed=rows)
    if V == 5003:
        _run(rows, 1, V, 384, seed=rows)


@pytest.mark.parametrize("rows", [1, 9, 16, 17, 32, 40])
@pytest.mark.parametrize("H", [128, 256, 384, 512, 640, 1024, 1536, 1664, 2048, 2176, 2560, 4096])
def test_every_division_of_the_columns(rows, H):
    # fewer words of four tiles than waves, as many, more; whole and short last words
    _run(rows, 1, 517, H, seed=rows + H)


def test_wide_vocabulary_and_rows():
    # checked at the first, the last and some other vocabulary rows
    import torch
    import markov_draft_sampling_amd as mds
    V, H = 151936 + 5, 512
    g = torch.Generator().manual_seed(1)
    codes = torch.randint(0, 256, (V, H // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(118, 123, (V, H // 32), generator=g, dtype=torch.uint8)
    tiled, ts = mds.tile_lm_head_mxfp4(codes.cuda(), scales.cuda())
    at = np.unique(np.concatenate([np.arange(140), np.arange(V - 140, V), np.random.default_rng(V).integers(0, V, 400)]))
    c = codes.numpy()[at]
    w = lr.mx_values(np.stack([c & 15, c >> 4], -1).reshape(len(at), H), scales.numpy()[at])
    x = torch.randn((224, H), generator=g).to(torch.bfloat16)
    for rows in (1, 7, 20, 64, 100, 224):
        print(f"4-bit LM head rows {rows} V {V} H {H}", flush=True)
        out = torch.full((rows, 1, V), 7.25, device="cuda")
        mds.lm_head_mxfp4(x[:rows].cuda(), tiled, ts, out, 1)
        _check(out[:, 0].cpu().numpy()[:, at].astype(np.float64), x[:rows].double().numpy(), w)


def test_a_matrix_past_32_bits():
    # 4.5 GB of codes: checked at the first and the last rows
    import torch
    import markov_draft_sampling_amd as mds
    V, H = 1100003, 8192
    g = torch.Generator(device="cuda").manual_seed(2)
    codes = torch.randint(0, 256, (V, H // 2), generator=g, dtype=torch.uint8, device="cuda")
    scales = torch.randint(116, 121, (V, H // 32), generator=g, dtype=torch.uint8, device="cuda")
    tiled, ts = mds.tile_lm_head_mxfp4(codes, scales)
    at = torch.cat([torch.arange(40), torch.arange(V - 40, V)])
    c = codes[at.cuda()].cpu().numpy()
    w = lr.mx_values(np.stack([c & 15, c >> 4], -1).reshape(80, H), scales[at.cuda()].cpu().numpy())
    del codes, scales
    x = torch.randn((40, H), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    for rows in (3, 40):
        out = torch.full((rows, 1, V), 7.25, device="cuda")
        mds.lm_head_mxfp4(x[:rows].cuda(), tiled, ts, out, 1)
        _check(out[:, 0, at.cuda()].cpu().numpy().astype(np.float64), x[:rows].double().numpy(), w)
    back = mds.unpack_lm_head_mxfp4(tiled, ts, V)
    assert torch.equal(back[at.cuda()].cpu().double(), torch.from_numpy(w))
    t2, s2 = mds.quantize_lm_head_mxfp4(back)  # (values of the format come back as they are, with scales that fit)
    assert torch.equal(mds.unpack_lm_head_mxfp4(t2, s2, V), back)


def test_outputs_strided_with_rows_left_alone():
    _run(6, 8, 1003, 256, seed=1, out_dtype="bf16", pad=5, extra=2)
    _run(6, 8, 1003, 256, seed=1, pad=5, extra=2)
    _run(6, 8, 1004, 256, seed=2, out_dtype="bf16", pad=4)
    _run(1, 3, 1004, 640, seed=2, out_dtype="bf16", pad=4)
    _run(1, 1, 1003, 640, seed=2, pad=3, extra=1)


@pytest.mark.parametrize("V,H", [(2, 128), (16, 512), (300, 256), (1003, 640), (77, 1920)])
def test_codes_scales_and_their_order(V, H):
    import torch
    import markov_draft_sampling_amd as mds
    for mode in ("quantize", "tile"):
        w, codes, scales, tiled, ts = _matrix(V, H, V, mode)
        want, want_s = lr.mx_tiles(codes, scales)
        assert np.array_equal(tiled.cpu().numpy(), want) and np.array_equal(ts.cpu().numpy(), want_s), mode
        back = mds.unpack_lm_head_mxfp4(tiled, ts, V)
        assert torch.equal(back.cpu().double(), torch.from_numpy(w))
        out = torch.full((V + 1, H), 7.0, dtype=torch.bfloat16, device="cuda")
        mds.unpack_lm_head_mxfp4(tiled, ts, out=out[:V])
        assert torch.equal(out[:V], back) and (out[V:] == 7).all()


def test_every_bf16_magnitude_is_quantised():
    # blocks of 32 from 2^-133 to the largest, ties of every code among them, and those that hold no number
    import torch
    import markov_draft_sampling_amd as mds
    H = 128
    top = np.arange(0x0000, 0x7F80, 5, dtype=np.uint16)
    bits = np.zeros((len(top), 4, 32), np.uint16)
    rng = np.random.default_rng(0)
    bits[:, :, 0] = top[:, None]
    below = np.maximum(top.astype(np.int64)[:, None, None] - rng.integers(0, 700, (len(top), 4, 31)), 0)
    bits[:, :, 1:] = below | (rng.integers(0, 2, below.shape) << 15)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0], np.float32)
    for i, e in enumerate(range(-60, 60)):
        t = torch.from_numpy(np.concatenate([ties, -ties]) * np.float32(2.0 ** e)).to(torch.bfloat16)
        bits[i * 7, 0, :16] = t.view(torch.int16).numpy().view(np.uint16)
        bits[i * 7, 0, 16:] = 0
    w = torch.from_numpy(bits.reshape(len(top), H).view(np.int16)).view(torch.bfloat16)
    codes, scales = lr.mx_quantize(w.float().numpy())
    tiled, ts = mds.quantize_lm_head_mxfp4(w.cuda())
    want, want_s = lr.mx_tiles(codes, scales)
    assert np.array_equal(ts.cpu().numpy(), want_s)
    assert np.array_equal(tiled.cpu().numpy(), want)
    bad = torch.ones((16, 128), dtype=torch.bfloat16)
    bad[3, 40], bad[5, 127], bad[9, 0] = float("nan"), float("inf"), -float("inf")
    back = mds.unpack_lm_head_mxfp4(*mds.quantize_lm_head_mxfp4(bad.cuda())).cpu()
    none = torch.zeros((16, 128), dtype=torch.bool)
    none[3, 32:64], none[5, 96:], none[9, :32] = True, True, True
    assert back[none].isnan().all() and (back[~none] == 1).all()


def test_scales_from_the_smallest_to_none():
    # every scale byte: logits of a unit vector are the weights themselves, bf16's range and NaN among them
    import torch
    import markov_draft_sampling_amd as mds
    H = 128
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, H // 16))
    scales = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, H // 32))
    tiled, ts = mds.tile_lm_head_mxfp4(torch.from_numpy(lr.mx_pack(codes)).cuda(), torch.from_numpy(scales).cuda())
    w = torch.from_numpy(lr.mx_values(codes, scales)).to(torch.bfloat16)
    back = mds.unpack_lm_head_mxfp4(tiled, ts, 256).cpu()
    assert torch.equal(back.isnan(), w.isnan()) and torch.equal(back.nan_to_num(0.0), w.nan_to_num(0.0))
    finite = torch.from_numpy(scales[:, 0] < 253)
    for rows in (1, 40):
        x = torch.zeros((rows, H), dtype=torch.bfloat16)
        x[:, 37] = 1.0
        out = torch.zeros((rows, 1, 256), device="cuda")
        mds.lm_head_mxfp4(x.cuda(), tiled, ts, out, 1)
        o = out[:, 0].cpu()
        assert (o[:, finite] == w[finite, 37].float()).all()
        assert o[:, 255].isnan().all()


def test_a_row_that_is_no_number_stays_alone():
    import torch
    import markov_draft_sampling_amd as mds
    w, _, _, tiled, ts = _matrix(200, 256, 3, "tile")
    for rows in (9, 50):
        x = torch.randn((rows, 256), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
        out, clean = torch.zeros((rows, 1, 200), device="cuda"), torch.zeros((rows, 1, 200), device="cuda")
        mds.lm_head_mxfp4(x, tiled, ts, clean, 1)
        x[4, 100] = float("nan")
        x[rows - 1, 0] = float("inf")
        mds.lm_head_mxfp4(x, tiled, ts, out, 1)
        o, c = out[:, 0].cpu(), clean[:, 0].cpu()
        keep = [r for r in range(rows) if r not in (4, rows - 1)]
        assert o[4].isnan().all() and not o[rows - 1].isfinite().any()
        assert torch.equal(o[keep], c[keep])


def test_other_streams_and_a_graph():
    import torch
    import markov_draft_sampling_amd as mds
    bits = torch.randn((1000, 512), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    tiled, ts = mds.quantize_lm_head_mxfp4(bits, stream=side)
    back = mds.unpack_lm_head_mxfp4(tiled, ts, 1000, stream=side)
    side.synchronize()
    t2, s2 = mds.quantize_lm_head_mxfp4(bits)
    assert torch.equal(tiled, t2) and torch.equal(ts, s2) and torch.equal(back, mds.unpack_lm_head_mxfp4(t2, s2, 1000))
    for rows in (3, 70):
        x = torch.randn((rows, 512), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
        out, want = torch.zeros((rows, 1, 1000), device="cuda"), torch.zeros((rows, 1, 1000), device="cuda")
        torch.cuda.synchronize()
        mds.lm_head_mxfp4(x, tiled, ts, out, 1, stream=side)
        side.synchronize()
        mds.lm_head_mxfp4(x, tiled, ts, want, 1)
        assert torch.equal(out, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mds.lm_head_mxfp4(x, tiled, ts, out, 1)
        for i in range(3):
            x.mul_(-1.25)
            g.replay()
            mds.lm_head_mxfp4(x, tiled, ts, want, 1)
            torch.cuda.synchronize()
            assert torch.equal(out, want), (rows, i)


def test_refusals_of_the_binding():
    import torch
    import markov_draft_sampling_amd as mds
    _, _, _, tiled, ts = _matrix(200, 256, 3, "tile")
    x = torch.zeros((6, 256), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((2, 3, 200), device="cuda")
    ok = dict(hidden=x, lm_head=tiled, scales=ts, out=out, K=3)
    mds.lm_head_mxfp4(**ok)
    for bad in (dict(hidden=x.float()), dict(hidden=x[:, ::2]), dict(hidden=x[:5]), dict(lm_head=tiled[:-1]),
                dict(lm_head=tiled.view(torch.int8)), dict(scales=ts[:, :128]), dict(scales=ts.cpu()),
                dict(out=out.half()), dict(out=out[:1]), dict(out=out[:, :2]), dict(K=4), dict(K=0),
                dict(out=out[..., ::2]), dict(hidden=x[:, :128])):
        with pytest.raises(mds.MdsError):
            mds.lm_head_mxfp4(**{**ok, **bad})
    for call, args in ((mds.quantize_lm_head_mxfp4, (x.float(),)), (mds.quantize_lm_head_mxfp4, (x[:, :100],)),
                       (mds.quantize_lm_head_mxfp4, (x[:, :128],)), (mds.quantize_lm_head_mxfp4, (x, tiled)),
                       (mds.tile_lm_head_mxfp4, (tiled.float(), ts)), (mds.tile_lm_head_mxfp4, (tiled, ts)),
                       (mds.unpack_lm_head_mxfp4, (tiled, ts, 300)), (mds.unpack_lm_head_mxfp4, (tiled, ts[:2])),
                       (mds.unpack_lm_head_mxfp4, (tiled, ts, 200, x))):
        with pytest.raises(mds.MdsError):
            call(*args)
