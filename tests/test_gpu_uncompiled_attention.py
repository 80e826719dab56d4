"""Attention called without the module of the compiled calls, on the GPU: the
same bits and the same refusals as with it."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu


def _set(cache, hnd=False):
    import torch
    g = torch.Generator().manual_seed(0)
    kp, vp = (torch.randn((40, 16, 2, 128), generator=g) for _ in range(2))
    if hnd:
        kp, vp = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (kp, vp))
    kind = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    a = dict(q=torch.randn((16, 4, 128), generator=g).to(torch.bfloat16).cuda(), k_pages=kp.to(kind).cuda(),
             v_pages=vp.to(kind).cuda(), block_table=torch.randperm(40, generator=g).view(2, 20).int().cuda(),
             query_start=t([0, 8, 15]), seq_lens=t([300, 317]), max_q_len=8, max_seq_len=317)
    if cache == "e4m3":
        a.update(k_scale=torch.tensor([0.5, 0.25]).cuda(), v_scale=torch.tensor([2.0, 1.5]).cuda())
    return a


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("more", [dict(), dict(window=50, sinks=7), dict(window=20), dict(causal=False, scale=0.3),
                                  dict(idx_map=True), dict(stream=True), dict(workspace=True)])
def test_equal_bits(cache, more, monkeypatch):
    import torch
    import markov_draft_sampling_amd as mds
    from markov_draft_sampling_amd import _serving
    a = {**_set(cache, hnd=True), **more}
    if "idx_map" in more:
        a["idx_map"] = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    if "stream" in more:
        a["stream"] = torch.cuda.Stream()
    if "workspace" in more:
        a["workspace"] = mds.new_workspace(mds.paged_attention_workspace_bytes(16, 2, 4, 2, 128, 8, 317))
    outs = []
    for compiled in (True, False):
        if not compiled:
            monkeypatch.setattr(_serving, "_calls", lambda needed=True: None)
        out, lse = torch.full_like(a["q"], 7.0), torch.full((16, 4), 7.0, device="cuda")
        torch.cuda.synchronize()
        ws = mds.paged_attention(out=out, lse=lse, **a)
        torch.cuda.synchronize()
        assert mds.workspace_status(ws) == 0
        outs.append((out, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert (outs[1][0][:15] != 7).any() and (outs[1][0][15:] == 7).all()


def test_the_same_refusals(monkeypatch):
    import torch
    import markov_draft_sampling_amd as mds
    from markov_draft_sampling_amd import _serving
    a = _set("bf16")
    a["out"] = torch.zeros_like(a["q"])
    bad = [dict(q=a["q"].float()), dict(q=a["q"][..., ::2]), dict(out=a["out"][:3]), dict(out=a["out"].cpu()),
           dict(k_pages=a["k_pages"].float()), dict(v_pages=a["v_pages"][:3]), dict(block_table=a["block_table"].long()),
           dict(block_table=a["block_table"][0]), dict(query_start=a["query_start"][:2]), dict(seq_lens=a["seq_lens"].cpu()),
           dict(max_q_len=-1), dict(max_q_len=1 << 40), dict(max_seq_len=-1), dict(scale=float("nan")), dict(window=-3),
           dict(sinks=-3), dict(k_scale=torch.ones(2).cuda()), dict(lse=torch.zeros(3).cuda()),
           dict(idx_map=a["block_table"]), dict(workspace=torch.zeros(256).cuda()),
           dict(workspace=torch.zeros(64, dtype=torch.uint8).cuda())]
    for compiled in (True, False):
        if not compiled:
            monkeypatch.setattr(_serving, "_calls", lambda needed=True: None)
        mds.paged_attention(**a)
        for b in bad:
            with pytest.raises(mds.MdsError):
                mds.paged_attention(**{**a, **b})
