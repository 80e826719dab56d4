"""The serving operators around drafting and verification, as cases that can be timed and compared.

Four operators, each in two forms on the same inputs: elementary torch
operations (``own = False``) and the library's calls (``own = True``).

* page tables: the paged cache's block tables, slot map and positions of the
  next chunk of tokens, from the requests' lengths and the last verification's
  accepted counts (``kv_page_tables``);
* append: a chunk's keys and values into the pages of the slot map
  (``kv_append``), bf16 or e4m3 pages;
* attention: a chunk of new tokens of every request over its paged cache
  (``paged_attention``): one token, the K + 1 tokens that verification scores,
  a draft block that attends both ways, a chunk of a prompt;
* 8-bit LM head: logits of B * K rows from an e4m3 matrix with one scale for
  each block of 128 x 128, the hidden rows quantised in blocks of 128
  (``lm_head_fp8``).
"""
from __future__ import annotations

import math

import torch

own = False

E4M3_MAX = 448.0
E4M3_FLOOR = 2.0 ** -100  # least amax of a quantisation block
DEV = "cuda"


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one decode step of 32 requests of 8 tokens (K = 7 drafts and the anchor), most of them inside their pages
        {"name": "tables_verify_b32", "op": "tables", "batch": 32, "slots": 48, "page": 16, "max_pages": 513,
         "ctx_lo": 1, "ctx_hi": 8192, "chunk_lo": 8, "chunk_hi": 8, "long_every": 0, "release_every": 0, "tight": False},
        # a mixed step of 1024 requests: verification chunks, a prompt chunk in every 64, finished requests released,
        # more tokens than pages for the last few
        {"name": "tables_mixed_b1024", "op": "tables", "batch": 1024, "slots": 1500, "page": 64, "max_pages": 520,
         "ctx_lo": 0, "ctx_hi": 32000, "chunk_lo": 0, "chunk_hi": 8, "long_every": 64, "release_every": 9, "tight": True},
        # the keys and values of a verification step of 32 requests into an 8-bit cache
        {"name": "append_verify_e4m3_b32", "op": "append", "tokens": 256, "kv_heads": 8, "dim": 128, "page": 16,
         "pages": 64, "cache": "e4m3", "padded": 0},
        # a prompt chunk of 16384 tokens, some rows padding
        {"name": "append_prompt_bf16", "op": "append", "tokens": 16384, "kv_heads": 8, "dim": 128, "page": 64,
         "pages": 320, "cache": "bf16", "padded": 37},
        # one request, one token: the latency of plain decoding
        {"name": "attend_single_b1", "op": "attention", "batch": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "chunk_lo": 1, "chunk_hi": 1, "ctx_lo": 1037, "ctx_hi": 1037, "cache": "bf16", "causal": True, "window": 0,
         "padded": 0},
        # verification of K = 7 drafts of 32 requests, ragged contexts
        {"name": "attend_verify_b32", "op": "attention", "batch": 32, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "chunk_lo": 8, "chunk_hi": 8, "ctx_lo": 100, "ctx_hi": 8192, "cache": "bf16", "causal": True, "window": 0,
         "padded": 0},
        # the same of 128 requests over an 8-bit cache, eight query heads a key head
        {"name": "attend_verify_e4m3_b128", "op": "attention", "batch": 128, "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 32, "chunk_lo": 8, "chunk_hi": 8, "ctx_lo": 1, "ctx_hi": 4096, "cache": "e4m3", "causal": True,
         "window": 0, "padded": 24},
        # the draft model's block of 7 query tokens, every one seeing the whole block
        {"name": "attend_block_b8_d64", "op": "attention", "batch": 8, "heads": 16, "kv_heads": 4, "dim": 64, "page": 64,
         "chunk_lo": 7, "chunk_hi": 7, "ctx_lo": 300, "ctx_hi": 2500, "cache": "bf16", "causal": False, "window": 0,
         "padded": 0},
        # a chunk of 2048 prompt tokens after 14000
        {"name": "attend_prompt_2048", "op": "attention", "batch": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "chunk_lo": 2048, "chunk_hi": 2048, "ctx_lo": 14000, "ctx_hi": 14000, "cache": "bf16", "causal": True,
         "window": 0, "padded": 0},
        # one long request under verification
        {"name": "attend_long_b1", "op": "attention", "batch": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "chunk_lo": 8, "chunk_hi": 8, "ctx_lo": 131072, "ctx_hi": 131072, "cache": "bf16", "causal": True, "window": 0,
         "padded": 0},
        # the draft LM head of one request on the V = 32000 configuration
        {"name": "lm_head_b1_v32000", "op": "lm_head", "batch": 1, "steps": 7, "vocab": 32000, "hidden": 4096,
         "out": "f32"},
        # the headline batch: 224 rows, V = 200064
        {"name": "lm_head_b32_v200064", "op": "lm_head", "batch": 32, "steps": 7, "vocab": 200064, "hidden": 4096,
         "out": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "attention", "attention", "attention", "lm_head"])
    if op == "tables":
        page = rng.choice([16, 32, 64, 128])
        batch = _log(rng, 1, 1024)
        hi = _log(rng, 1, 32000)
        return {"op": op, "batch": batch, "slots": batch + rng.randint(0, 500), "page": page,
                "max_pages": -(-(hi + 2048) // page) + rng.randint(1, 9), "ctx_lo": rng.randint(0, 1), "ctx_hi": hi,
                "chunk_lo": rng.randint(0, 1), "chunk_hi": rng.choice([1, 2, 5, 8, 17]),
                "long_every": rng.choice([0, 0, 16, 50]), "release_every": rng.choice([0, 7, 12]),
                "tight": rng.random() < 0.3}
    if op == "append":
        page = rng.choice([16, 32, 64, 128])
        cache = rng.choice(["bf16", "e4m3"])
        tokens = _log(rng, 1, 16384 if cache == "bf16" else 4000)
        return {"op": op, "tokens": tokens, "kv_heads": rng.choice([1, 2, 4, 5, 8]), "dim": rng.choice([64, 128]),
                "page": page, "pages": -(-tokens // page) + rng.randint(1, 20), "cache": cache,
                "padded": rng.choice([0, 1, 30])}
    if op == "attention":
        kv = rng.choice([1, 2, 4, 8])
        kind = rng.choice(["one", "verify", "verify", "block", "prompt"])
        c = {"op": op, "batch": 1, "heads": kv * rng.choice([1, 2, 3, 4, 8]), "kv_heads": kv,
             "dim": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128]), "chunk_lo": 1, "chunk_hi": 1,
             "ctx_lo": 0, "ctx_hi": 0, "cache": rng.choice(["bf16", "bf16", "e4m3"]), "causal": kind != "block",
             "window": 0, "padded": rng.choice([0, 0, 3, 40])}
        if kind == "prompt":
            c["batch"] = rng.randint(1, 2)
            c["chunk_hi"] = _log(rng, 33, 800)
            c["chunk_lo"] = rng.randint(1, c["chunk_hi"])
            c["ctx_hi"] = _log(rng, 1, 8000)
        else:
            c["batch"] = _log(rng, 1, 128)
            c["chunk_hi"] = 1 if kind == "one" else rng.randint(2, 17)
            c["chunk_lo"] = 1 if kind == "one" else rng.randint(0, c["chunk_hi"])
            c["ctx_hi"] = _log(rng, 1, min(65536, 250000 // c["batch"]))
        c["ctx_lo"] = rng.choice([0, 1, c["ctx_hi"]])
        if c["causal"] and rng.random() < 0.3:
            c["window"] = rng.choice([17, 128, 1000])
        return c
    vocab = rng.choice([4099, 32000, 50017, 100003, 151936])
    return {"op": op, "batch": _log(rng, 1, 32), "steps": rng.choice([1, 3, 7]), "vocab": vocab,
            "hidden": 128 * rng.randint(2, 32), "out": rng.choice(["f32", "f32", "bf16"])}


def _spread(n, lo, hi, salt):
    """n whole numbers over [lo, hi], the same for every seed (low-discrepancy), the last one hi."""
    v = [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + salt) % 1.0)) for i in range(n)]
    v[-1] = hi
    return v


def _attention_lengths(c):
    ctx = _spread(c["batch"], c["ctx_lo"], c["ctx_hi"], 0.37)
    chunk = _spread(c["batch"], c["chunk_lo"], c["chunk_hi"], 0.11)
    return ctx, chunk


def _pairs(ctx, chunk, causal, window):
    """(query, key) pairs that a request's mask leaves, and the keys read."""
    if not causal:
        return chunk * (ctx + chunk), (ctx + chunk if chunk else 0)
    n = 0
    for t in range(chunk):
        seen = ctx + t + 1
        n += min(seen, window) if window else seen
    lo = max(0, ctx + 1 - window) if window else 0
    return n, (ctx + chunk - lo if chunk else 0)


def work(case):
    c = case
    if c["op"] == "tables":
        ctx, chunk = _table_lengths(c)
        tokens = sum(x for x in chunk if x > 0)
        cap = _token_capacity(c)
        held = sum(-(-(a + max(x, 0)) // c["page"]) for a, x in zip(ctx, chunk)) // 4
        return {"bytes": 16 * cap + 4 * tokens // c["page"] + 44 * c["batch"] + 4 * min(held, tokens),
                "flops": 20 * (tokens + c["batch"])}
    if c["op"] == "append":
        n = c["tokens"] * c["kv_heads"] * c["dim"] * 2
        return {"bytes": n * 2 + n * (1 if c["cache"] == "e4m3" else 2) + 8 * (c["tokens"] + c["padded"]), "flops": n}
    if c["op"] == "attention":
        ctx, chunk = _attention_lengths(c)
        es = 1 if c["cache"] == "e4m3" else 2
        pairs = keys = 0
        for a, x in zip(ctx, chunk):
            p, k = _pairs(a, x, c["causal"], c["window"])
            pairs += p
            keys += k
        tokens = sum(chunk)
        return {"bytes": keys * c["kv_heads"] * c["dim"] * 2 * es + tokens * c["heads"] * (4 * c["dim"] + 4)
                + 4 * keys // c["page"], "flops": 4 * pairs * c["heads"] * c["dim"]}
    rows, V, H = c["batch"] * c["steps"], c["vocab"], c["hidden"]
    return {"bytes": V * H + 4 * -(-V // 128) * (H // 128) + rows * H * 2 + rows * V * (2 if c["out"] == "bf16" else 4),
            "flops": 2 * rows * V * H}


# ---------------------------------------------------------------- prepare --
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)
    s = {"tables": _prepare_tables, "append": _prepare_append, "attention": _prepare_attention,
         "lm_head": _prepare_lm_head}[case["op"]](case, g)
    s["case"] = case
    return s


def _table_lengths(c):
    """Lengths before the step and chunk lengths (-1: finished, its pages go back)."""
    ctx = _spread(c["batch"], c["ctx_lo"], c["ctx_hi"], 0.21)
    chunk = _spread(c["batch"], c["chunk_lo"], c["chunk_hi"], 0.83)
    if c["long_every"]:
        for i in range(c["long_every"] - 1, c["batch"], c["long_every"]):
            chunk[i] = 100 + (i * 977) % 1900
    if c["release_every"]:
        for i in range(c["release_every"] - 1, c["batch"], c["release_every"]):
            chunk[i] = -1
    return ctx, chunk


def _token_capacity(c):
    return sum(x for x in _table_lengths(c)[1] if x > 0) + 5


def _perm(n, g):
    return torch.randperm(n, generator=g, device=DEV)


def _prepare_tables(c, g):
    B, N, P, MP = c["batch"], c["slots"], c["page"], c["max_pages"]
    ctx, chunk = _table_lengths(c)
    # the last verification kept 1 + (0 .. 7) tokens of the chunk before: kv_len is that much less than the context
    acc = torch.randint(0, 8, (B,), generator=g, device=DEV, dtype=torch.int32)
    order = _perm(B, g)
    ctx_t = torch.tensor(ctx, device=DEV)[order]
    chunk_t = torch.tensor(chunk, device=DEV, dtype=torch.int32)[order]
    acc = torch.minimum(acc, (ctx_t - 1).clamp(min=0)).to(torch.int32)
    kv = (ctx_t - acc - 1).clamp(min=0)
    slot = _perm(N, g)[:B].to(torch.int32)
    idx_map = torch.where(torch.arange(B, device=DEV) % 97 == 96, torch.full_like(slot, -1), slot)
    kv_len = torch.zeros(N, device=DEV, dtype=torch.int32)
    kv_len[slot.long()] = kv.to(torch.int32)
    held = torch.zeros(N, device=DEV, dtype=torch.int32)
    # pages of the chunk before verification (8 tokens) are held already
    held[slot.long()] = torch.clamp((kv + 8 + P - 1) // P, max=MP).to(torch.int32)
    used = int(held.sum())
    need = sum(-(-max(x, 0) // P) + 1 for x in chunk)
    n_free = max(1, need // 4 if c["tight"] else need)
    n_pages = sum(min(MP, -(-(x + 8) // P)) for x in ctx) + need  # every seed's held pages and the free ones fit
    pages = _perm(n_pages, g).to(torch.int32)
    start = torch.cumsum(held, 0) - held
    col = torch.arange(MP, device=DEV)
    table = torch.where(col[None, :] < held[:, None], pages[(start[:, None] + col[None, :]).clamp(max=n_pages - 1)], 0)
    free = torch.zeros(n_pages, device=DEV, dtype=torch.int32)
    free[:n_free] = pages[used:used + n_free]
    T = _token_capacity(c)
    return {"kv_len": kv_len, "chunk_len": chunk_t, "block_table": table.to(torch.int32).contiguous(),
            "pages_held": held, "free_list": free, "advance": acc, "idx_map": idx_map,
            "free_count": torch.tensor([n_free], device=DEV, dtype=torch.int32),
            "query_start": torch.zeros(B + 1, device=DEV, dtype=torch.int32),
            "seq_lens": torch.zeros(B, device=DEV, dtype=torch.int32),
            "positions": torch.zeros(T, device=DEV, dtype=torch.int64),
            "slot_map": torch.zeros(T, device=DEV, dtype=torch.int64), "kv_len_out": kv_len.clone(),
            "pages_held_out": held.clone(), "free_count_out": torch.zeros(1, device=DEV, dtype=torch.int32),
            "status": torch.zeros(1, device=DEV, dtype=torch.int32)}


def _cache_dtype(c):
    return torch.float8_e4m3fn if c["cache"] == "e4m3" else torch.bfloat16


def _prepare_append(c, g):
    T, Hk, D, P, NP = c["tokens"], c["kv_heads"], c["dim"], c["page"], c["pages"]
    rows = T + c["padded"]
    k = torch.randn((rows, Hk, D), generator=g, device=DEV).to(torch.bfloat16)
    v = torch.randn((rows, Hk, D), generator=g, device=DEV).to(torch.bfloat16)
    slot = torch.full((rows,), -1, device=DEV, dtype=torch.int64)
    # chunks of 8 tokens in a row, as requests have them, somewhere in the pool
    n8 = -(-T // 8)
    base = _perm(NP * P // 8, g)[:n8] * 8
    slot[:T] = (base[:, None] + torch.arange(8, device=DEV)[None, :]).reshape(-1)[:T]
    s = {"k": k, "v": v, "slot_map": slot, "k_scale": None, "v_scale": None}
    for n in ("k_pages", "v_pages"):
        s[n] = torch.randn((NP, P, Hk, D), generator=g, device=DEV).to(_cache_dtype(c))
    if c["cache"] == "e4m3":
        s["k_scale"] = 0.01 + 0.02 * torch.rand(Hk, generator=g, device=DEV)
        s["v_scale"] = 0.01 + 0.02 * torch.rand(Hk, generator=g, device=DEV)
    return s


def _prepare_attention(c, g):
    B, Hq, Hk, D, P = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    ctx, chunk = _attention_lengths(c)
    seq = [a + x for a, x in zip(ctx, chunk)]
    held = [-(-x // P) for x in seq]
    NP = sum(held) + 3
    order = _perm(NP, g).to(torch.int32)
    MP = max(held) + 2
    start = torch.tensor([sum(held[:i]) for i in range(B)] if B < 512 else [0], device=DEV)
    held_t = torch.tensor(held, device=DEV)
    col = torch.arange(MP, device=DEV)
    table = torch.where(col[None, :] < held_t[:, None], order[(start[:, None] + col[None, :]).clamp(max=NP - 1)], 0)
    T = sum(chunk)
    gain = 0.5 + 2.0 * torch.rand((1, Hq, 1), generator=g, device=DEV)  # diffuse and peaked heads
    q = (torch.randn((T + c["padded"], Hq, D), generator=g, device=DEV) * gain).to(torch.bfloat16)
    s = {"q": q, "k_scale": None, "v_scale": None, "block_table": table.to(torch.int32).contiguous()}
    amp = 1.0
    if c["cache"] == "e4m3":
        amp = 60.0
        s["k_scale"] = (0.9 + 0.2 * torch.rand(Hk, generator=g, device=DEV)) / amp
        s["v_scale"] = (0.9 + 0.2 * torch.rand(Hk, generator=g, device=DEV)) / amp
    for n in ("k_pages", "v_pages"):
        x = torch.randn((NP, P, Hk, D), generator=g, device=DEV, dtype=torch.bfloat16)
        s[n] = x if amp == 1.0 else (x.float() * amp).clamp(-E4M3_MAX, E4M3_MAX).to(_cache_dtype(c))
        del x
    qs = [0]
    for x in chunk:
        qs.append(qs[-1] + x)
    s["query_start"] = torch.tensor(qs, device=DEV, dtype=torch.int32)
    s["seq_lens"] = torch.tensor(seq, device=DEV, dtype=torch.int32)
    s["out"] = torch.zeros((T + c["padded"], Hq, D), device=DEV, dtype=torch.bfloat16)
    s["lse"] = torch.zeros((T + c["padded"], Hq), device=DEV, dtype=torch.float32)
    s["tokens"], s["max_q_len"], s["max_seq_len"] = T, max(chunk), max(seq)
    s["workspace"] = None
    # what the dense plain form indexes by: request and place of every token
    s["of"] = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(chunk, device=DEV))
    s["at"] = torch.arange(T, device=DEV) - s["query_start"][:-1].long()[s["of"]]
    return s


def _prepare_lm_head(c, g):
    V, H, rows = c["vocab"], c["hidden"], c["batch"] * c["steps"]
    hidden = torch.randn((rows, H), generator=g, device=DEV)
    hidden[:, torch.randint(0, H, (8,), generator=g, device=DEV)] *= 12.0  # outlier channels
    VB, HB = -(-V // 128), H // 128
    w = torch.zeros((VB * 128, H), device=DEV, dtype=torch.bfloat16)
    w[:V].normal_(0.0, 3.0 / math.sqrt(H), generator=g)
    blocks = w.view(VB, 128, HB, 128)
    amax = blocks.abs().amax(dim=(1, 3)).float()
    scales = (torch.clamp(amax, min=E4M3_FLOOR) / E4M3_MAX).contiguous()
    codes = torch.empty((VB * 128, H), device=DEV, dtype=torch.float8_e4m3fn)
    for i in range(0, VB, 256):  # in pieces: the float32 copy is large
        codes.view(VB, 128, HB, 128)[i:i + 256] = (blocks[i:i + 256].float() / scales[i:i + 256, None, :, None]).to(
            torch.float8_e4m3fn)
    del w, blocks
    # the order in which the library keeps the matrix: tiles of 16 rows by 128 columns, in each 8 x 16 pieces of 16
    VT = -(-V // 16)
    tiled = codes[: VT * 16].view(torch.uint8).view(VT, 16, HB, 8, 16).permute(0, 2, 3, 1, 4).contiguous().view(VT, 16 * H)
    dt = torch.bfloat16 if c["out"] == "bf16" else torch.float32
    return {"hidden": hidden.to(torch.bfloat16), "codes": codes, "scales": scales,
            "tiled": tiled.view(torch.float8_e4m3fn), "workspace": None,
            "out": torch.zeros((c["batch"], c["steps"], V), device=DEV, dtype=dt)}


# -------------------------------------------------------------------- run --
def run(state):
    if own:
        return _run_own(state)
    return {"tables": _plain_tables, "append": _plain_append, "attention": _plain_attention,
            "lm_head": _plain_lm_head}[state["case"]["op"]](state)


def _run_own(s):
    import markov_draft_sampling_amd as mds
    c = s["case"]
    if c["op"] == "tables":
        mds.kv_page_tables(s["kv_len"], s["chunk_len"], s["block_table"], s["pages_held"], s["free_list"],
                           s["free_count"], c["page"], s["query_start"], s["seq_lens"], s["positions"], s["slot_map"],
                           s["kv_len_out"], s["pages_held_out"], s["free_count_out"], status=s["status"],
                           idx_map=s["idx_map"], advance=s["advance"], advance_add=1)
        return _table_outputs(s, s["block_table"], s["free_list"])
    if c["op"] == "append":
        mds.kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["slot_map"], k_scale=s["k_scale"],
                      v_scale=s["v_scale"])
        return _append_outputs(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
    if c["op"] == "attention":
        s["workspace"] = mds.paged_attention(
            s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["query_start"], s["seq_lens"], s["out"],
            s["max_q_len"], s["max_seq_len"], causal=c["causal"], window=c["window"], k_scale=s["k_scale"],
            v_scale=s["v_scale"], lse=s["lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    s["workspace"] = mds.lm_head_fp8(s["hidden"], s["tiled"], s["scales"], s["out"], c["steps"],
                                     workspace=s["workspace"])
    return s["out"]


def _table_outputs(s, table, free):
    return {"query_start": s["query_start"], "seq_lens": s["seq_lens"], "positions": s["positions"],
            "slot_map": s["slot_map"], "kv_len": s["kv_len_out"], "pages_held": s["pages_held_out"],
            "free_count": s["free_count_out"], "block_table": table, "free_list": free}


def _append_outputs(k, v, k_scale, v_scale):
    if k_scale is None:
        return {"k_pages": k, "v_pages": v}
    return {"k_pages": k.float() * k_scale[:, None], "v_pages": v.float() * v_scale[:, None]}


# ------------------------------------------------------------ plain forms --
def _plain_tables(s):
    c = s["case"]
    P, MP = c["page"], c["max_pages"]
    N, T, NP = s["kv_len"].numel(), s["positions"].numel(), s["free_list"].numel()
    i64 = torch.int64
    slot = s["idx_map"].to(i64)
    live = (slot >= 0) & (slot < N)
    row = torch.where(live, slot, 0)
    chunk = s["chunk_len"].to(i64)
    held = s["pages_held"].to(i64)[row]
    done = live & (chunk < 0)
    here = live & (chunk >= 0)
    ctx = s["kv_len"].to(i64)[row] + s["advance"].to(i64) + 1
    n = torch.where(here, chunk, 0)
    end = torch.cumsum(n, 0)
    first = end - n
    want = (ctx + n + P - 1) // P
    fits = here & (want <= MP) & (end <= T)
    need = torch.where(fits, (want - held).clamp(min=0), 0)
    upto = torch.cumsum(need, 0)
    # pages of finished requests go back first, in batch order
    back = torch.where(done, held, 0)
    back_end = torch.cumsum(back, 0)
    count = s["free_count"].to(i64)
    i = torch.arange(NP, device=slot.device)
    j = i - count
    b = torch.searchsorted(back_end, j.clamp(min=0), right=True).clamp(max=slot.numel() - 1)
    given = s["block_table"].to(i64)[row[b], (j - back_end[b] + back[b]).clamp(0, MP - 1)]
    free = torch.where((j >= 0) & (j < back_end[-1]), given, s["free_list"].to(i64))
    avail = count + back_end[-1]
    granted = fits & ((need == 0) | (upto <= avail))
    taken = torch.where(granted, upto, 0).amax()
    # page i of the new ones comes from the end of the free list
    b = torch.searchsorted(upto, i, right=True).clamp(max=slot.numel() - 1)
    at = (row[b] * MP + held[b] + i - upto[b] + need[b]).clamp(0, N * MP - 1)
    page = free[(avail - 1 - i).clamp(min=0)]
    table = torch.cat([s["block_table"].reshape(-1).to(i64), page[:1]])
    table[torch.where(i < taken, at, N * MP)] = page
    table = table[:-1].view(N, MP)
    t = torch.arange(T, device=slot.device)
    b = torch.searchsorted(end, t, right=True).clamp(max=slot.numel() - 1)
    inside = (t < end[-1]) & here[b]
    pos = torch.where(inside, ctx[b] + t - first[b], 0)
    of_page = table[row[b], (pos // P).clamp(max=MP - 1)]
    slot_map = torch.where(inside & granted[b], of_page * P + pos % P, -1)
    kv_out = torch.cat([s["kv_len"].to(i64), ctx[:1]])
    kv_out[torch.where(live, slot, N)] = torch.where(done, 0, ctx)
    held_out = torch.cat([s["pages_held"].to(i64), ctx[:1]])
    held_out[torch.where(live, slot, N)] = torch.where(done, 0, held + torch.where(granted, need, 0))
    i32 = torch.int32
    return {"query_start": torch.cat([first[:1], end]).to(i32),
            "seq_lens": torch.where(granted, ctx + n, 0).to(i32), "positions": pos, "slot_map": slot_map,
            "kv_len": kv_out[:-1].to(i32), "pages_held": held_out[:-1].to(i32),
            "free_count": (avail - taken).to(i32), "block_table": table.to(i32), "free_list": free.to(i32)}


def _plain_append(s):
    live = s["slot_map"] >= 0
    # a padding row writes what the first live row's slot gets anyway
    first = torch.argmax(live.to(torch.int32))
    src = torch.where(live, torch.arange(live.numel(), device=live.device), first)
    slot = s["slot_map"][src]

    def put(x, pages, scale):
        x = x.float()[src]
        if scale is not None:
            x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        new = pages.clone()
        new.view(-1, *pages.shape[2:]).view(torch.uint8 if scale is not None else pages.dtype)[slot] = x.to(
            pages.dtype).view(torch.uint8 if scale is not None else pages.dtype)
        return new

    return _append_outputs(put(s["k"], s["k_pages"], s["k_scale"]), put(s["v"], s["v_pages"], s["v_scale"]),
                           s["k_scale"], s["v_scale"])


def _plain_attention(s):
    """Dense over the batch: every request padded to the longest chunk and the longest context."""
    c = s["case"]
    B, Hq, Hk, D, P = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    T, N, L, G = s["tokens"], s["max_q_len"], s["max_seq_len"], c["heads"] // c["kv_heads"]
    dev = s["q"].device
    if T == 0:
        return {"out": torch.zeros_like(s["out"]), "lse": torch.zeros_like(s["lse"])}
    seq = s["seq_lens"].long()
    chunk = s["query_start"].long().diff()
    key = torch.arange(L, device=dev)
    page = s["block_table"].long()[:, key // P]  # [B, L]
    at = page * P + key % P

    def gather(pages, scale):
        # codes are gathered as bytes: indexing knows no 8-bit floating point
        x = pages.view(-1, Hk, D)
        x = (x.view(torch.uint8)[at].view(pages.dtype) if scale is not None else x[at]).float()
        x = x if scale is None else x * scale[:, None]
        return x.transpose(1, 2).contiguous().view(B * Hk, L, D)

    q = torch.zeros((B, N, Hq, D), device=dev)
    q[s["of"], s["at"]] = s["q"][:T].float()
    q = q.view(B, N, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B * Hk, N * G, D)
    x = torch.bmm(q, gather(s["k_pages"], s["k_scale"]).transpose(1, 2)).view(B, Hk, N, G, L)
    x *= 1.0 / math.sqrt(D)
    pos = (seq - chunk)[:, None] + torch.arange(N, device=dev)[None, :]  # [B, N]
    seen = (key[None, None, :] < seq[:, None, None]).expand(B, N, L)
    if c["causal"]:
        seen = seen & (key[None, None, :] <= pos[:, :, None])
    if c["window"]:
        seen = seen & (key[None, None, :] > pos[:, :, None] - c["window"])
    x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x -= top
    x.exp_()
    total = x.sum(dim=-1, keepdim=True)
    o = torch.bmm(x.view(B * Hk, N * G, L), gather(s["v_pages"], s["v_scale"])).view(B, Hk, N, G, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + torch.log(total))[..., 0]
    out = torch.zeros_like(s["out"])
    out[:T] = o.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D)[s["of"], s["at"]].to(out.dtype)
    lse_out = torch.zeros_like(s["lse"])
    lse_out[:T] = lse.permute(0, 2, 1, 3).reshape(B, N, Hq)[s["of"], s["at"]]
    return {"out": out, "lse": lse_out}


def _plain_lm_head(s):
    c = s["case"]
    V, H = c["vocab"], c["hidden"]
    HB = H // 128
    x = s["hidden"].float().view(-1, HB, 128)
    sx = x.abs().amax(dim=-1, keepdim=True).clamp(min=E4M3_FLOOR)
    sx = sx / torch.full_like(sx, E4M3_MAX)  # a true quotient: by a number, torch multiplies by its reciprocal
    x = ((x / sx).to(torch.float8_e4m3fn).float() * sx).view(-1, H)
    w = s["codes"].float().view(-1, 128, HB, 128) * s["scales"][:, None, :, None]
    z = x @ w.view(-1, H)[:V].t()
    return z.view(c["batch"], c["steps"], V).to(s["out"].dtype)


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    """The operators' definitions in 64 bits, request by request and block by block."""
    if case["op"] == "tables":
        return None  # whole numbers: nothing to round
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "lm_head": _exact_lm_head}[case["op"]](case, s)


def _e4m3_values():
    v = torch.arange(127, dtype=torch.float64)
    e, m = torch.div(v, 8, rounding_mode="floor"), v % 8
    return torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7))


def _round_e4m3(x):
    """float64 to the nearest e4m3 value, ties to the even code, past the largest to the largest."""
    val = _e4m3_values().to(x.device)
    a = x.abs().clamp(max=E4M3_MAX)
    hi = torch.searchsorted(val, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = val[hi] - a, a - val[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(val[code], x)


def _exact_append(c, s):
    out = {}
    for n in ("k", "v"):
        scale = s[n + "_scale"]
        pages = s[n + "_pages"].float().double()
        flat = pages.view(-1, c["kv_heads"], c["dim"])
        x = s[n][: c["tokens"]].double()
        if scale is not None:
            sc = scale.double()[None, :, None]
            flat *= sc
            x = _round_e4m3((x / sc).float().double()) * sc  # the quotient is a float32 one
        flat[s["slot_map"][: c["tokens"]]] = x
        out[n + "_pages"] = pages
    return out


def _exact_attention(c, s):
    Hk, G, P = c["kv_heads"], c["heads"] // c["kv_heads"], c["page"]
    ctx, chunk = _attention_lengths(c)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    t0 = 0
    for b, (a, n) in enumerate(zip(ctx, chunk)):
        if n == 0:
            continue
        L = a + n
        pages = s["block_table"][b, : -(-L // P)].long()
        for h in range(Hk):
            k = s["k_pages"][:, :, h][pages].float().double().reshape(-1, c["dim"])[:L]
            v = s["v_pages"][:, :, h][pages].float().double().reshape(-1, c["dim"])[:L]
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for i in range(0, n, 512):  # rows in pieces, so that the scores fit
                m = min(512, n - i)
                q = s["q"][t0 + i:t0 + i + m, h * G:(h + 1) * G].double().reshape(m * G, -1)
                x = (q @ k.t()) / math.sqrt(c["dim"])
                at = (a + i + torch.arange(m, device=DEV)).repeat_interleave(G)[:, None]
                key = torch.arange(L, device=DEV)[None, :]
                if c["causal"]:
                    x[key > at] = -math.inf
                if c["window"]:
                    x[key <= at - c["window"]] = -math.inf
                z = torch.logsumexp(x, dim=-1, keepdim=True)
                x -= z
                x.exp_()
                out[t0 + i:t0 + i + m, h * G:(h + 1) * G] = (x @ v).view(m, G, -1)
                lse[t0 + i:t0 + i + m, h * G:(h + 1) * G] = z.view(m, G)
        t0 += n
    return {"out": out, "lse": lse}


def _exact_lm_head(c, s):
    V, H = c["vocab"], c["hidden"]
    z = torch.zeros((c["batch"] * c["steps"], V), dtype=torch.float64, device=DEV)
    for h in range(0, H, 128):  # one block of 128 columns at a time
        x = s["hidden"][:, h:h + 128].double()
        sx = (x.abs().amax(dim=-1, keepdim=True).clamp(min=E4M3_FLOOR) / E4M3_MAX).float().double()
        x = _round_e4m3((x / sx).float().double()) * sx  # the quotient is a float32 one
        w = s["codes"][:V, h:h + 128].float().double() * s["scales"][:, h // 128].double().repeat_interleave(128)[:V, None]
        z += x @ w.t()
    return z.view(c["batch"], c["steps"], V)
