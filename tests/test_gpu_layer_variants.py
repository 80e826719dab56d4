"""Every variant of the kernels of a layer's step that a call can take, on the
GPU, at remainders of its tiles (the sizes: layer_cases.py)."""
from __future__ import annotations

import pytest

import layer_cases as lc
import layer_ref as lr

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
