"""Plain references of the operators of a layer's step for the tests, in
float64 and request by request, sharing no code with the library: norm and
rotation, attention with a window and first tokens that stay visible, the
microscaled 4-bit format."""
from __future__ import annotations

import math

import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def norm_rope(x, weight, eps, positions, inv_freq, interleaved, rope_scale):
    """float64 (out, e) of x [T, heads, D] (CPU, bf16 values): e bounds what float32 arithmetic on the way
    may be off, before the rounding of what is written.

    y = x r w with r = 1 / sqrt(ss / D + eps): the float32 sum of D squares is within (D + 1) 2^-24 of itself, which
    the root halves; quotient, sum, root, reciprocal and the two products add at most 2^-24 each. Turned, each of the
    two terms takes the error of its y, of cosine and sine (2^-21: four units in the last place of sincospi, the
    rounding of the half turn, the product with rope_scale) and of two roundings; the angle is float64 to within 2^-51 of itself."""
    x = x.double()
    T, _, D = x.shape
    y, rel = x, 0.0
    if weight is not None:
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + eps) * weight.double()
        rel = (D / 2 + 8) * 2.0 ** -24
    out, err = y.clone(), y.abs() * rel
    if inv_freq is not None and inv_freq.numel():
        half = inv_freq.numel()
        first = torch.arange(half) * 2 if interleaved else torch.arange(half)
        second = first + 1 if interleaved else first + half
        a = positions.double()[:, None] * inv_freq.double()[None, :]
        c, s = (torch.cos(a) * rope_scale)[:, None, :], (torch.sin(a) * rope_scale)[:, None, :]
        p, q = y[..., first], y[..., second]
        out[..., first], out[..., second] = p * c - q * s, q * c + p * s
        e = (p.abs() + q.abs()) * abs(rope_scale) * (rel + 2.0 ** -21 + 2.0 ** -23 + (a.abs() * 2.0 ** -51)[:, None, :])
        err[..., first], err[..., second] = e, e
    return out, err


def attention_sinks(q, k_pages, v_pages, table, query_start, seq_lens, scale, causal, window, sinks, idx_map=None,
                    k_scale=None, v_scale=None):
    """float64 (out, lse, A, S, seen pages): A = sum p |v|, S = scale * max_j sum |q k|. CPU tensors, caches as values.
    seen pages: for each request the pages of which some token sees a key."""
    T, Hq, D = q.shape
    P, Hk = k_pages.shape[1], k_pages.shape[2]
    G = Hq // Hk
    out, A = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    lse, S = torch.full((T, Hq), -math.inf, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    pages = []
    for b in range(len(seq_lens)):
        t0, t1, L = int(query_start[b]), int(query_start[b + 1]), int(seq_lens[b])
        s = b if idx_map is None else int(idx_map[b])
        pages.append(set())
        if s < 0 or L <= 0 or t1 == t0:
            continue
        key = torch.arange(L)
        pos = (L - (t1 - t0) + torch.arange(t1 - t0))[:, None]
        seen = (key <= pos) if causal else torch.ones(t1 - t0, L, dtype=torch.bool)
        if window:
            seen = seen & ((key > pos - window) | (key < sinks))
        at = key[seen.any(0)]
        seen = seen[:, seen.any(0)]
        pages[b] = set((at // P).tolist())
        slot = [int(table[s][p // P]) * P + p % P for p in at.tolist()]
        for h in range(Hq):
            k = k_pages.reshape(-1, Hk, D)[slot, h // G].double()
            v = v_pages.reshape(-1, Hk, D)[slot, h // G].double()
            if k_scale is not None:
                k, v = k * float(k_scale[h // G]), v * float(v_scale[h // G])
            x = (q[t0:t1, h].double() @ k.T) * scale
            x[~seen] = -math.inf
            z = torch.logsumexp(x, 1)
            w = torch.where(seen, torch.exp(x - torch.where(z == -math.inf, 0.0, z)[:, None]), 0.0)
            out[t0:t1, h], A[t0:t1, h], lse[t0:t1, h] = w @ v, w @ v.abs(), z
            S[t0:t1, h] = torch.where(seen, q[t0:t1, h].double().abs() @ k.abs().T, 0.0).amax(1) * scale
    return out, lse, A, S, pages


def mx_quantize(w):
    """float32 [V, H] (bf16 values): (codes 0 .. 15 [V, H], scale bytes [V, H / 32]) by the microscaling rule."""
    V, H = w.shape
    x = np.asarray(w, np.float64).reshape(V, H // 32, 32)
    amax = np.maximum(np.abs(x).max(-1), 2.0 ** -100)
    e = np.frexp(amax)[1] - 1 - 2
    y = np.abs(x) / np.exp2(e.astype(np.float64))[..., None]
    grid = E2M1[:8]
    hi = np.clip(np.searchsorted(grid, np.minimum(y, 6.0)), 0, 7)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - np.minimum(y, 6.0), np.minimum(y, 6.0) - grid[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code + 8 * np.signbit(x)).reshape(V, H).astype(np.uint8), (e + 127).astype(np.uint8)


def mx_values(codes, scales):
    """float64 weights of codes 0 .. 15 [V, H] and scale bytes [V, H / 32]."""
    s = scales.astype(np.float64)
    unit = np.where(s == 255, np.nan, np.exp2(s - 127))
    return E2M1[codes] * np.repeat(unit, 32, axis=1)


def mx_tiles(codes, scales):
    """The tiled arrays of the two, element by element from the stated index."""
    V, H = codes.shape
    vt, G = -(-V // 16), -(-H // 512)
    tiled, ts = np.zeros(vt * 8 * H, np.uint8), np.zeros(vt * 256 * G, np.uint8)
    v, c = np.meshgrid(np.arange(V), np.arange(H), indexing="ij")
    at = ((v // 16) * (H // 128) + c // 128) * 1024 + ((c % 128) // 32) * 256 + (v % 16) * 16 + (c % 32) // 2
    np.bitwise_or.at(tiled, at.ravel(), (codes << (4 * (c % 2)).astype(np.uint8)).ravel())
    v, c = np.meshgrid(np.arange(V), np.arange(0, H, 32), indexing="ij")
    ts[((v // 16) * G + c // 512) * 256 + ((c % 128) // 32) * 64 + (v % 16) * 4 + (c % 512) // 128] = scales
    return tiled.reshape(vt, 8 * H), ts.reshape(vt, 256 * G)


def mx_pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
