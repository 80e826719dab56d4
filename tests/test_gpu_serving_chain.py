"""The serving operators together, as a serving loop runs them around drafting
and verification: page tables from the last accepted counts, append, attention
over the pages, the 8-bit LM head, then the draft loop and verification on its
logits; several steps, a prompt chunk and a finished request among them, each
step's attention checked against a plain recomputation over the whole history,
and the same step as a captured graph."""
from __future__ import annotations

import math

import numpy as np
import pytest

import serving_ref as sr

pytestmark = pytest.mark.gpu

B, K, HK, G, D, P, V, H = 5, 3, 2, 2, 64, 16, 2000, 256
HQ = HK * G


class Loop:
    def __init__(self, cache):
        import torch
        import markov_draft_sampling_amd as mds
        self.mds, self.torch = mds, torch
        g = torch.Generator().manual_seed(4)
        z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        self.n_slots, self.max_pages, self.n_pages, self.T = B + 2, 12, 40, 80
        self.kv_len, self.held, self.count = z(self.n_slots), z(self.n_slots), z(1) + self.n_pages
        self.table, self.free = z(self.n_slots, self.max_pages), torch.arange(self.n_pages, dtype=torch.int32).cuda()
        self.qs, self.seq, self.status = z(B + 1), z(B), z(1)
        self.pos, self.slot = z(self.T, dt=torch.int64), z(self.T, dt=torch.int64)
        dt = torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn
        self.kp, self.vp = z(self.n_pages, P, HK, D, dt=torch.float32).to(dt), z(self.n_pages, P, HK, D, dt=torch.float32).to(dt)
        self.ks = self.vs = None
        if cache == "e4m3":
            self.ks, self.vs = torch.full((HK,), 0.02, device="cuda"), torch.full((HK,), 0.03, device="cuda")
        self.idx = torch.tensor([3, 0, 6, 1, 5], dtype=torch.int32, device="cuda")
        self.chunk, self.adv = z(B), z(B)
        self.q, self.k, self.v = (z(self.T, n, D, dt=torch.bfloat16) for n in (HQ, HK, HK))
        self.out, self.lse = torch.zeros_like(self.q), z(self.T, HQ, dt=torch.float32)
        self.mix = (torch.randn((HQ * D, H), generator=g) / math.sqrt(HQ * D)).cuda()
        self.head, self.scales = mds.quantize_lm_head_fp8((torch.randn((V, H), generator=g) * 0.3).to(torch.bfloat16).cuda())
        self.hidden = z(B * (K + 1), H, dt=torch.bfloat16)
        self.target = z(B, K + 1, V, dt=torch.float32)
        self.ws = mds.new_workspace(mds.paged_attention_workspace_bytes(self.T, B, HQ, HK, D, self.T, self.max_pages * P))
        self.head_ws = mds.new_workspace(mds.lm_head_fp8_workspace_bytes(B, K + 1, V, H))
        self.g = g
        self.history = [([], []) for _ in range(B)]  # what a plain cache would hold, per request

    def fill(self, n):
        for t in (self.q, self.k, self.v):
            t.copy_(self.torch.randn(t.shape, generator=self.g).to(self.torch.bfloat16))

    def step(self, add):
        m = self.mds
        m.kv_page_tables(self.kv_len, self.chunk, self.table, self.held, self.free, self.count, P, self.qs, self.seq,
                         self.pos, self.slot, self.kv_len, self.held, self.count, status=self.status, idx_map=self.idx,
                         advance=self.adv, advance_add=add)
        m.kv_append(self.k, self.v, self.kp, self.vp, self.slot, k_scale=self.ks, v_scale=self.vs, status=self.status)
        m.paged_attention(self.q, self.kp, self.vp, self.table, self.qs, self.seq, self.out, self.T, self.max_pages * P,
                          idx_map=self.idx, k_scale=self.ks, v_scale=self.vs, lse=self.lse, workspace=self.ws)

    def check(self, chunk, kept):
        """The step's outputs against the history: kept[b] tokens of the last chunk stayed."""
        torch = self.torch
        kc, vc = self.k.cpu(), self.v.cpu()
        as_cache = lambda x, s: x.double() if s is None else torch.from_numpy(  # noqa: E731
            sr.e4m3_round((x.float() / s.cpu()[:, None]).numpy())) * s.cpu()[:, None].double()
        t0 = 0
        out, lse = self.out.cpu(), self.lse.cpu()
        for b in range(B):
            hk, hv = self.history[b]
            n = chunk[b]
            if n < 0:
                hk.clear()
                hv.clear()
                assert int(self.seq[b]) == 0
                continue
            ctx = kept[b]
            del hk[ctx:], hv[ctx:]
            for t in range(t0, t0 + n):
                hk.append(as_cache(kc[t], self.ks))
                hv.append(as_cache(vc[t], self.vs))
            L = ctx + n
            assert int(self.seq[b]) == L and self.pos[t0:t0 + n].tolist() == list(range(ctx, L))
            if n == 0:
                continue
            pages = -(-L // P)
            kk = torch.zeros(pages * P, HK, D, dtype=torch.float64)
            vv = torch.zeros_like(kk)
            kk[:L], vv[:L] = torch.stack(hk), torch.stack(hv)
            ref = sr.attention(self.q.cpu()[t0:t0 + n], kk.view(pages, P, HK, D), vv.view(pages, P, HK, D),
                               [list(range(pages))], [0, n], [L], 1 / math.sqrt(D))
            tol, ltol = sr.attention_tolerance(ref[0], ref[2], ref[3], D, L)
            assert ((out[t0:t0 + n].double() - ref[0]).abs() <= tol).all()
            assert ((lse[t0:t0 + n].double() - ref[1]).abs() <= ltol).all()
            t0 += n


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_serving_loop(cache):
    import torch
    import markov_draft_sampling_amd as mds
    lp = Loop(cache)
    rng = np.random.default_rng(1)
    seeds = torch.arange(B, dtype=torch.int64, device="cuda")
    temp = torch.full((B,), 0.8, device="cuda")
    temp[1] = 0.0
    w1 = (torch.randn(V, 32, generator=lp.g) * 0.05).to(torch.bfloat16).cuda()
    w2 = (torch.randn(V, 32, generator=lp.g) * 0.05).to(torch.bfloat16).cuda()
    chunk, kept, acc = [7, 20, 1, 12, 5], [0] * B, None
    for step in range(6):
        lp.chunk.copy_(torch.tensor(chunk, dtype=torch.int32))
        lp.adv.copy_(torch.tensor([0] * B if acc is None else acc, dtype=torch.int32))
        lp.fill(sum(max(c, 0) for c in chunk))
        lp.step(0)
        torch.cuda.synchronize()
        assert int(lp.status.item()) == 0 and mds.workspace_status(lp.ws) == 0
        lp.check(chunk, kept)
        # the scores of every request's last K + 1 rows, drafts from them, and what verification keeps
        rows = torch.tensor([max(0, int(lp.qs[b + 1]) - K - 1 + j) for b in range(B) for j in range(K + 1)]).cuda()
        lp.hidden.copy_((lp.out.view(lp.T, -1)[rows].float() @ lp.mix).to(torch.bfloat16))
        mds.lm_head_fp8(lp.hidden, lp.head, lp.scales, lp.target, K + 1, workspace=lp.head_ws)
        cache_l = torch.empty((B, K, V), device="cuda")
        toks = torch.empty((B, K), dtype=torch.int32, device="cuda")
        lse = torch.empty((B, K), device="cuda")
        anchor, apos = torch.arange(B, dtype=torch.int32).cuda(), torch.full((B,), 10 + step, dtype=torch.int64).cuda()
        mds.markov_draft_loop(lp.target, w1, w2, anchor, apos, temp, seeds, cache_l, toks, lse)
        out_t = torch.empty((B, K + 1), dtype=torch.int32, device="cuda")
        n_acc = torch.empty(B, dtype=torch.int32, device="cuda")
        mds.rejection_verify(lp.target.view(B * (K + 1), V), cache_l, toks, temp, seeds, apos, out_t, n_acc, draft_lse=lse)
        torch.cuda.synchronize()
        accepted = n_acc.tolist()
        assert all(0 <= a <= K for a in accepted)
        # prompts keep every token, verification chunks the anchor and the accepted drafts
        acc = [0 if c < 0 else c if c != K + 1 else accepted[b] + 1 for b, c in enumerate(chunk)]
        kept = [0 if c < 0 else kp + a for kp, a, c in zip(kept, acc, chunk)]
        chunk = [K + 1] * B
        if step == 2:
            chunk[3] = -1  # finished
        if step == 3:
            chunk[3] = 9   # a new request in its slot
        if step == 4:
            chunk[0] = 0   # nothing new this time
    del rng


def test_the_step_as_a_graph():
    import torch
    lp, eager = Loop("bf16"), Loop("bf16")
    for x in (lp, eager):
        x.chunk.fill_(K + 1)
    g = torch.cuda.CUDAGraph()
    warm = Loop("bf16")
    warm.chunk.fill_(K + 1)
    warm.step(1)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        lp.step(1)
    for i in range(5):
        a = torch.tensor([-1 if i == 0 else (i + b) % (K + 1) for b in range(B)], dtype=torch.int32)
        for x in (lp, eager):
            x.adv.copy_(a)
            x.g.manual_seed(i)
            x.fill(0)
        g.replay()
        eager.step(1)
        torch.cuda.synchronize()
        for n in ("out", "lse", "table", "kv_len", "held", "count", "slot", "pos", "seq", "kp", "vp"):
            assert torch.equal(getattr(lp, n), getattr(eager, n)), (i, n)
    assert int(lp.status.item()) == 0
