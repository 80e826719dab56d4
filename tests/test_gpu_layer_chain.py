"""A layer's step as a serving loop runs it: page tables, norm and rotation
with the append, attention with a window and first tokens that stay visible,
the 4-bit LM head, then drafting and verification on its logits, over several
steps, with pages between the two visible parts given away; each step against
a plain recomputation over the whole history; and the same step as a captured
graph."""
from __future__ import annotations

import math

import numpy as np
import pytest

import layer_ref as lr
import serving_ref as sr

pytestmark = pytest.mark.gpu

B, K, HK, G, D, R, P, V, H, W, S = 4, 3, 2, 3, 64, 32, 16, 1500, 256, 24, 4
HQ = HK * G


class Loop:
    def __init__(self):
        import torch
        import markov_draft_sampling_amd as mds
        self.mds, self.torch = mds, torch
        self.g = torch.Generator().manual_seed(4)
        z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        self.n_slots, self.max_pages, self.n_pages, self.T = B + 1, 12, 48, 90
        self.kv_len, self.held, self.count = z(self.n_slots), z(self.n_slots), z(1) + self.n_pages
        self.table, self.free = z(self.n_slots, self.max_pages), torch.arange(self.n_pages, dtype=torch.int32).cuda()
        self.qs, self.seq, self.status = z(B + 1), z(B), z(1)
        self.pos, self.slot = z(self.T, dt=torch.int64), z(self.T, dt=torch.int64)
        self.kp, self.vp = (z(self.n_pages, P, HK, D, dt=torch.bfloat16) for _ in range(2))
        self.idx = torch.tensor([3, 0, 4, 1], dtype=torch.int32, device="cuda")
        self.chunk, self.adv = z(B), z(B)
        self.qkv = z(self.T, HQ + 2 * HK, D, dt=torch.bfloat16)
        self.q, self.out, self.lse = z(self.T, HQ, D, dt=torch.bfloat16), z(self.T, HQ, D, dt=torch.bfloat16), \
            z(self.T, HQ, dt=torch.float32)
        self.freq, self.rs = mds.rope_frequencies(R, scaling="yarn", factor=4.0, trained_len=64)
        self.qw, self.kw = ((1 + 0.2 * torch.randn(D, generator=self.g)).to(torch.bfloat16).cuda() for _ in range(2))
        self.mix = (torch.randn((HQ * D, H), generator=self.g) / math.sqrt(HQ * D)).cuda()
        self.head = mds.quantize_lm_head_mxfp4((torch.randn((V, H), generator=self.g) * 0.3).to(torch.bfloat16).cuda())
        self.hidden, self.target = z(B * (K + 1), H, dt=torch.bfloat16), z(B, K + 1, V, dt=torch.float32)
        self.ws = mds.new_workspace(mds.paged_attention_workspace_bytes(self.T, B, HQ, HK, D, self.T, self.max_pages * P, W, S))

    def fill(self):
        self.qkv.copy_(self.torch.randn(self.qkv.shape, generator=self.g).to(self.torch.bfloat16))

    def step(self, add):
        m, x = self.mds, self.qkv
        m.kv_page_tables(self.kv_len, self.chunk, self.table, self.held, self.free, self.count, P, self.qs, self.seq,
                         self.pos, self.slot, self.kv_len, self.held, self.count, status=self.status, idx_map=self.idx,
                         advance=self.adv, advance_add=add)
        m.qk_norm_rope_append(x[:, :HQ], x[:, HQ:HQ + HK], x[:, HQ + HK:], self.pos, self.freq, self.q, self.kp, self.vp,
                              self.slot, q_weight=self.qw, k_weight=self.kw, rope_scale=self.rs, status=self.status)
        m.paged_attention(self.q, self.kp, self.vp, self.table, self.qs, self.seq, self.out, self.T, self.max_pages * P,
                          idx_map=self.idx, window=W, sinks=S, lse=self.lse, workspace=self.ws)


def test_a_serving_loop():
    import torch
    import markov_draft_sampling_amd as mds
    lp = Loop()
    w = mds.unpack_lm_head_mxfp4(*lp.head, V).cpu().double().numpy()
    seeds = torch.arange(B, dtype=torch.int64, device="cuda")
    temp = torch.tensor([0.8, 0.0, 0.8, 1.0], device="cuda")
    w1, w2 = ((torch.randn(V, 32, generator=lp.g) * 0.05).to(torch.bfloat16).cuda() for _ in range(2))
    history = [([], []) for _ in range(B)]
    chunk, kept, acc = [40, 20, 1, 29], [0] * B, [0] * B
    for step in range(8):
        lp.chunk.copy_(torch.tensor(chunk, dtype=torch.int32))
        lp.adv.copy_(torch.tensor(acc, dtype=torch.int32))
        lp.fill()
        lp.step(0)
        torch.cuda.synchronize()
        assert int(lp.status.item()) == 0 and mds.workspace_status(lp.ws) == 0
        x, q, out = lp.qkv.cpu(), lp.q.cpu(), lp.out.cpu()
        pos = lp.pos.cpu()
        qr, qe = lr.norm_rope(x[:, :HQ], lp.qw.cpu(), 1e-6, pos, lp.freq.cpu(), False, lp.rs)
        kr, ke = lr.norm_rope(x[:, HQ:HQ + HK], lp.kw.cpu(), 1e-6, pos, lp.freq.cpu(), False, lp.rs)
        assert ((q.double() - qr).abs() <= 2.0 ** -8 * qr.abs() + 1.01 * qe + 1e-37).all()
        pages_k, pages_v = lp.kp.cpu(), lp.vp.cpu()
        table = lp.table.cpu()
        t0 = 0
        for b in range(B):
            hk, hv = history[b]
            del hk[kept[b]:], hv[kept[b]:]
            n, L = chunk[b], kept[b] + chunk[b]
            assert int(lp.seq[b]) == L and pos[t0:t0 + n].tolist() == list(range(kept[b], L))
            for t in range(t0, t0 + n):  # what the pages got, within its rounding, and from then on as it is
                p, s = int(pos[t]), int(lp.idx[b])
                at = int(table[s][p // P]), p % P
                assert ((pages_k[at].double() - kr[t]).abs() <= 2.0 ** -8 * kr[t].abs() + 1.01 * ke[t] + 1e-37).all()
                assert torch.equal(pages_v[at], x[t, HQ + HK:])
                hk.append(pages_k[at])
                hv.append(pages_v[at])
            if n:
                np_ = -(-L // P)
                kk, vv = torch.zeros(np_ * P, HK, D), torch.zeros(np_ * P, HK, D)
                kk[:L], vv[:L] = torch.stack(hk).float(), torch.stack(hv).float()
                ref, z, A, Sx, seen = lr.attention_sinks(q[t0:t0 + n], kk.view(np_, P, HK, D), vv.view(np_, P, HK, D),
                                                         [list(range(np_))], [0, n], [L], 1 / math.sqrt(D), True, W, S)
                tol, ltol = sr.attention_tolerance(ref, A, Sx, D, L)
                assert ((out[t0:t0 + n].double() - ref).abs() <= tol).all()
                assert ((lp.lse.cpu()[t0:t0 + n].double() - z).abs() <= ltol).all()
                # a page that no later token sees either goes to somebody else
                for p in range(-(-S // P), max(0, (kept[b] + 1 - W) // P)):
                    lp.kp[table[int(lp.idx[b])][p]] = float("nan")
                    lp.vp[table[int(lp.idx[b])][p]] = float("nan")
            t0 += n
        rows = torch.tensor([max(0, int(lp.qs[b + 1]) - K - 1 + j) for b in range(B) for j in range(K + 1)]).cuda()
        lp.hidden.copy_((lp.out.view(lp.T, -1)[rows].float() @ lp.mix).to(torch.bfloat16))
        mds.lm_head_mxfp4(lp.hidden, *lp.head, lp.target, K + 1)
        h = lp.hidden.cpu().double().numpy()
        err = np.abs(lp.target.cpu().numpy().reshape(-1, V) - h @ w.T)
        assert (err <= (4 * H / 32 + 16) * 2.0 ** -24 * (np.abs(h) @ np.abs(w).T) + 1e-37).all()
        cache_l, toks = torch.empty((B, K, V), device="cuda"), torch.empty((B, K), dtype=torch.int32, device="cuda")
        lse = torch.empty((B, K), device="cuda")
        anchor, apos = torch.arange(B, dtype=torch.int32).cuda(), torch.full((B,), 10 + step, dtype=torch.int64).cuda()
        mds.markov_draft_loop(lp.target, w1, w2, anchor, apos, temp, seeds, cache_l, toks, lse)
        out_t, n_acc = torch.empty((B, K + 1), dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
        mds.rejection_verify(lp.target.view(B * (K + 1), V), cache_l, toks, temp, seeds, apos, out_t, n_acc, draft_lse=lse)
        torch.cuda.synchronize()
        accepted = n_acc.tolist()
        # prompts keep every token, verification chunks the anchor and the accepted drafts
        acc = [c if c != K + 1 else accepted[b] + 1 for b, c in enumerate(chunk)]
        kept = [kp + a for kp, a in zip(kept, acc)]
        chunk = [K + 1] * B
        if step == 2:
            chunk[2] = 30  # a prompt's next part beside the others


def test_the_step_as_a_graph():
    import torch
    lp, eager, warm = Loop(), Loop(), Loop()
    for x in (lp, eager, warm):
        x.chunk.fill_(K + 1)
    warm.step(1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lp.step(1)
        lp.mds.lm_head_mxfp4(lp.hidden, *lp.head, lp.target, K + 1)
    for i in range(6):
        a = torch.tensor([-1 if i == 0 else (i + b) % (K + 1) for b in range(B)], dtype=torch.int32)
        for x in (lp, eager):
            x.adv.copy_(a)
            x.g.manual_seed(i)
            x.fill()
            x.hidden.copy_(torch.randn(x.hidden.shape, generator=x.g).to(torch.bfloat16))
        g.replay()
        eager.step(1)
        eager.mds.lm_head_mxfp4(eager.hidden, *eager.head, eager.target, K + 1)
        torch.cuda.synchronize()
        for n in ("q", "out", "lse", "table", "kv_len", "held", "count", "slot", "pos", "seq", "kp", "vp", "target"):
            assert torch.equal(getattr(lp, n), getattr(eager, n)), (i, n)
    assert int(lp.status.item()) == 0
