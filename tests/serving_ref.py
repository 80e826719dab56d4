"""Plain references of the serving operators for the tests: request by request
in Python and float64, sharing no code with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

E4M3_VALUES = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                        for e in range(16) for m in range(8)][:127])


def e4m3_round(x):
    """float32 array -> the nearest e4m3 values (float64), ties to the even
    code, past 448 to 448; NaN stays."""
    x = np.asarray(x, np.float32).astype(np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(E4M3_VALUES, np.nan_to_num(a)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3_VALUES[hi] - a, a - E4M3_VALUES[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.where(np.isnan(x), np.nan, np.copysign(E4M3_VALUES[code], x))


class TableState:
    """A page allocator's state and the step of mds_kv_page_tables on it."""

    def __init__(self, n_slots, max_pages, page, n_pages, free):
        self.P, self.n_pages = page, n_pages
        self.kv_len = [0] * n_slots
        self.held = [0] * n_slots
        self.table = [[-1] * max_pages for _ in range(n_slots)]
        self.free = list(free) + [-7] * (n_pages - len(free))
        self.count = len(free)

    def step(self, chunk, idx_map=None, advance=None, advance_add=0, max_tokens=64):
        B, N, P = len(chunk), len(self.kv_len), self.P
        mp = len(self.table[0])
        idx = list(range(B)) if idx_map is None else list(idx_map)
        status = 0
        slots = []
        for b in range(B):
            s = idx[b]
            if s >= N or (s >= 0 and idx.count(s) > 1):
                status |= 8
                s = -1
            slots.append(s)
        for b in range(B):  # finished requests first
            s = slots[b]
            if s >= 0 and chunk[b] < 0:
                for i in range(self.held[s]):
                    if self.count < self.n_pages:
                        self.free[self.count] = self.table[s][i]
                        self.count += 1
                    else:
                        status |= 8
                self.held[s] = self.kv_len[s] = 0
        qs, seq, pos, slot = [0], [], [], []
        asked = taken = 0
        for b in range(B):
            s = slots[b]
            n = chunk[b] if s >= 0 and chunk[b] >= 0 else 0
            first = sum(chunk[i] for i in range(b) if slots[i] >= 0 and chunk[i] > 0)
            end = first + n
            qs.append(min(end, max_tokens))
            if s < 0 or chunk[b] < 0:
                seq.append(0)
                continue
            ctx = self.kv_len[s] + (advance[b] + advance_add if advance is not None else 0)
            self.kv_len[s] = ctx
            want = -(-(ctx + n) // P)
            fits = want <= mp and end <= max_tokens
            need = max(0, want - self.held[s]) if fits else 0
            asked += need
            ok = fits and (need == 0 or asked <= self.count)
            if not ok:
                status |= 32
            else:
                for i in range(need):
                    self.table[s][self.held[s] + i] = self.free[self.count - 1 - (asked - need) - i]
                self.held[s] += need
                if need:
                    taken = asked
            seq.append(ctx + n if ok else 0)
            for i in range(n):
                if first + i < max_tokens:
                    p = ctx + i
                    pos.append(p)
                    slot.append(self.table[s][p // P] * P + p % P if ok else -1)
        self.count -= taken
        pos += [0] * (max_tokens - len(pos))
        slot += [-1] * (max_tokens - len(slot))
        return dict(query_start=qs, seq_lens=seq, positions=pos, slot_map=slot, status=status)


def attention(q, k_pages, v_pages, table, query_start, seq_lens, scale, causal=True, window=0, idx_map=None,
              k_scale=None, v_scale=None):
    """float64 (out, lse, A, S): A = sum p |v| and S = scale * max_j sum |q k|,
    the scales of the rounding errors. CPU tensors, caches already as values."""
    T, Hq, D = q.shape
    Hk = k_pages.shape[2]
    P = k_pages.shape[1]
    G = Hq // Hk
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    A = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    S = torch.zeros(T, Hq, dtype=torch.float64)
    for b in range(len(seq_lens)):
        t0, t1, L = int(query_start[b]), int(query_start[b + 1]), int(seq_lens[b])
        s = b if idx_map is None else int(idx_map[b])
        if s < 0 or L <= 0:
            continue
        at = [int(table[s][p // P]) * P + p % P for p in range(L)]
        for h in range(Hq):
            k = k_pages.reshape(-1, Hk, D)[at, h // G].double()
            v = v_pages.reshape(-1, Hk, D)[at, h // G].double()
            if k_scale is not None:
                k, v = k * float(k_scale[h // G]), v * float(v_scale[h // G])
            for t in range(t0, t1):
                p = L - (t1 - t0) + (t - t0)
                hi = min(L, p + 1) if causal else L
                lo = max(0, p - window + 1) if window else 0
                if hi <= lo:
                    continue
                qq = q[t, h].double()
                x = (k[lo:hi] @ qq) * scale
                z = torch.logsumexp(x, 0)
                w = torch.exp(x - z)
                out[t, h] = w @ v[lo:hi]
                A[t, h] = w @ v[lo:hi].abs()
                lse[t, h] = z
                S[t, h] = (k[lo:hi].abs() @ qq.abs()).max() * scale
    return out, lse, A, S


def attention_tolerance(ref, A, S, D, L):
    """Bounds of |out - ref| and |lse - ref|: the scores are float32 sums of D
    exact products (and a few roundings of x itself), which moves p by at most
    twice that; p is rounded to bf16 (half a step: 2^-8), sums over L keys in
    float32, the exponential within 2^-21, out rounded to bf16."""
    x = (D + 8) * 2.0 ** -24 * S
    rel = 2 * x + 2 * L * 2.0 ** -24 + 2.0 ** -20
    return 2.0 ** -8 * ref.abs() + (2.0 ** -8 * 1.01 + rel)[..., None] * A + 1e-30, x + L * 2.0 ** -24 + 2.0 ** -20


def quantize_blocks(w, rows, cols):
    """float32 [R, C] in blocks of rows x cols: (e4m3 values float64, scales
    float32), the last block of rows may be short."""
    R, C = w.shape
    rb = -(-R // rows)
    scales = np.zeros((rb, C // cols), np.float32)
    q = np.zeros((R, C))
    for i in range(rb):
        for j in range(C // cols):
            blk = w[i * rows:(i + 1) * rows, j * cols:(j + 1) * cols].astype(np.float32)
            s = np.float32(max(np.abs(blk).max(), np.float32(2.0 ** -100)) / np.float32(448.0))
            scales[i, j] = s
            q[i * rows:(i + 1) * rows, j * cols:(j + 1) * cols] = e4m3_round(blk / s)
    return q, scales


def lm_head(xq, xs, wq, ws):
    """float64 logits and sum of magnitudes from e4m3 values and block scales."""
    z = a = 0
    for j in range(xs.shape[1]):
        x = xq[:, j * 128:(j + 1) * 128] * xs[:, j:j + 1].astype(np.float64)
        w = wq[:, j * 128:(j + 1) * 128] * np.repeat(ws[:, j].astype(np.float64), 128)[: wq.shape[0], None]
        z = z + x @ w.T
        a = a + np.abs(x) @ np.abs(w).T
    return z, a
