"""A layer's step between its projections and the logits, as cases that can be timed and compared.

Three operators, each in two forms on the same inputs: elementary torch
operations (``own = False``) and the library's calls (``own = True``).

* norm and rotation: the queries and keys of new tokens normed head by head
  and rotated by their positions, into output rows (``qk_norm_rope``) or, keys
  and values, into the pages of the cache (``qk_norm_rope_append``);
* attention over a paged cache with a sliding window and a few first tokens
  that stay visible (``paged_attention`` with ``window`` and ``sinks``);
* 4-bit LM head: e2m1 codes with a power-of-two scale for 32 columns of a row;
  a bf16 matrix brought to that form and back (``quantize_lm_head_mxfp4``,
  ``unpack_lm_head_mxfp4``), and logits of bf16 hidden rows (``lm_head_mxfp4``).
"""
from __future__ import annotations

import math

import torch

own = False

E4M3_MAX = 448.0
DEV = "cuda"


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one request decodes one token: nothing but latency
        {"name": "rope_append_one_token", "op": "rope", "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "norm": True, "interleaved": False, "factor": 1.0, "append": True, "cache": "bf16", "page": 16, "pages": 64,
         "padded": 0, "far": 30000},
        # the 8 tokens (K = 7 drafts and the anchor) of 32 requests, an 8-bit cache, angles scaled for long contexts
        {"name": "rope_append_verify_b32_e4m3", "op": "rope", "tokens": 256, "heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "norm": True, "interleaved": False, "factor": 8.0, "append": True, "cache": "e4m3", "page": 16,
         "pages": 40, "padded": 8, "far": 131072},
        # prompts of 16384 tokens in one step
        {"name": "rope_append_prompt_16k", "op": "rope", "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "norm": True, "interleaved": False, "factor": 1.0, "append": True, "cache": "bf16", "page": 64,
         "pages": 260, "padded": 0, "far": 16384},
        # half of each head rotated, neighbouring elements paired, no norm and no cache
        {"name": "rope_interleaved_partial_4k", "op": "rope", "tokens": 4099, "heads": 24, "kv_heads": 3, "dim": 64,
         "rot": 32, "norm": False, "interleaved": True, "factor": 4.0, "append": False, "cache": "bf16", "page": 16,
         "pages": 1, "padded": 0, "far": 1 << 20},
        # one token of one request, far behind its first tokens
        {"name": "sinks_one_token", "op": "attention", "batch": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "chunk_lo": 1, "chunk_hi": 1, "ctx_lo": 30000, "ctx_hi": 30000, "cache": "bf16", "window": 1024, "sinks": 4,
         "padded": 0},
        # verification of 32 requests in long chats
        {"name": "sinks_verify_b32", "op": "attention", "batch": 32, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "chunk_lo": 8, "chunk_hi": 8, "ctx_lo": 100, "ctx_hi": 32768, "cache": "bf16", "window": 4096, "sinks": 4,
         "padded": 0},
        # a full decoding batch over an 8-bit cache, 8 query heads a key head
        {"name": "sinks_decode_b128_e4m3", "op": "attention", "batch": 128, "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64, "chunk_lo": 1, "chunk_hi": 1, "ctx_lo": 1, "ctx_hi": 12000, "cache": "e4m3", "window": 2000,
         "sinks": 16, "padded": 0},
        # a chunk of a long prompt
        {"name": "sinks_prompt_2k", "op": "attention", "batch": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "chunk_lo": 2048, "chunk_hi": 2048, "ctx_lo": 14336, "ctx_hi": 14336, "cache": "bf16", "window": 4096,
         "sinks": 64, "padded": 0},
        # a checkpoint's matrix brought to 4 bits, and the values that it then has
        {"name": "mxfp4_quantize_v50017", "op": "quantize", "vocab": 50017, "hidden": 4096},
        # one request's next token
        {"name": "mxfp4_head_1row_v32000", "op": "lm_head", "batch": 1, "steps": 1, "vocab": 32000, "hidden": 2048,
         "out": "f32"},
        # the K = 7 rows of one request's draft
        {"name": "mxfp4_head_7rows_v200064", "op": "lm_head", "batch": 1, "steps": 7, "vocab": 200064, "hidden": 4096,
         "out": "f32"},
        # those of 32 requests
        {"name": "mxfp4_head_224rows_v151936", "op": "lm_head", "batch": 32, "steps": 7, "vocab": 151936, "hidden": 4096,
         "out": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "attention", "attention", "lm_head", "lm_head", "quantize"])
    if op == "rope":
        kv = rng.choice([1, 2, 3, 4, 8])
        dim = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
        heads = kv * rng.choice([1, 2, 3, 4, 8])
        page = rng.choice([16, 32, 64, 128])
        tokens = _log(rng, 1, max(2, min(16384, 16384 * 48 * 128 // ((heads + 2 * kv) * dim))))
        return {"op": op, "tokens": tokens, "heads": heads, "kv_heads": kv, "dim": dim,
                "rot": rng.choice([dim, dim, dim // 32 * 16, 16]), "norm": rng.random() < 0.6,
                "interleaved": rng.random() < 0.4, "factor": rng.choice([1.0, 1.0, 4.0, 32.0]),
                "append": rng.random() < 0.7, "cache": rng.choice(["bf16", "bf16", "e4m3"]), "page": page,
                "pages": -(-tokens // page) + rng.randint(1, 12), "padded": rng.choice([0, 1, 30]),
                "far": _log(rng, 100, 1 << 20)}
    if op == "attention":
        kv = rng.choice([1, 2, 4, 8])
        kind = rng.choice(["one", "one", "verify", "verify", "prompt"])
        c = {"op": op, "batch": 1, "heads": kv * rng.choice([1, 2, 3, 4, 8]), "kv_heads": kv,
             "dim": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128]), "chunk_lo": 1, "chunk_hi": 1,
             "ctx_lo": 0, "ctx_hi": 0, "cache": rng.choice(["bf16", "bf16", "e4m3"]), "window": _log(rng, 17, 4096),
             "sinks": rng.choice([1, 4, 4, 16, 63, 64, 100]), "padded": rng.choice([0, 0, 3, 40])}
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
        return c
    if op == "quantize":
        return {"op": op, "vocab": _log(rng, 300, 50017), "hidden": 128 * rng.randint(1, 32)}
    return {"op": op, "batch": _log(rng, 1, 32), "steps": rng.choice([1, 3, 7]),
            "vocab": rng.choice([4099, 32000, 50017, 100003, 151936]), "hidden": 128 * rng.randint(2, 32),
            "out": rng.choice(["f32", "f32", "bf16"])}


def _spread(n, lo, hi, salt):
    """n whole numbers over [lo, hi], the same for every seed (low-discrepancy), the last one hi."""
    v = [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + salt) % 1.0)) for i in range(n)]
    v[-1] = hi
    return v


def _attention_lengths(c):
    ctx = _spread(c["batch"], c["ctx_lo"], c["ctx_hi"], 0.37)
    chunk = _spread(c["batch"], c["chunk_lo"], c["chunk_hi"], 0.11)
    return ctx, chunk


def _pairs(ctx, chunk, window, sinks):
    """(query, key) pairs that a request's mask leaves, and the keys read."""
    n = 0
    for t in range(chunk):
        lo = max(0, ctx + t + 1 - window)
        n += ctx + t + 1 - lo + min(sinks, lo)
    lo = max(0, ctx + 1 - window)
    return n, (ctx + chunk - lo + min(sinks, lo) if chunk else 0)


def work(case):
    c = case
    if c["op"] == "rope":
        rows = c["tokens"] + (0 if c["append"] else c["padded"])
        q, k = (c["tokens"] + c["padded"]) * c["heads"] * c["dim"], rows * c["kv_heads"] * c["dim"]
        es = 1 if c["append"] and c["cache"] == "e4m3" else 2
        kv = (2 if c["append"] else 1) * k
        return {"bytes": 4 * q + (2 + es) * kv + (16 if c["append"] else 8) * (c["tokens"] + c["padded"])
                + 4 * c["rot"] + (4 * c["dim"] if c["norm"] else 0), "flops": (q + k) * (7 if c["norm"] else 3)}
    if c["op"] == "attention":
        ctx, chunk = _attention_lengths(c)
        es = 1 if c["cache"] == "e4m3" else 2
        pairs = keys = 0
        for a, x in zip(ctx, chunk):
            p, k = _pairs(a, x, c["window"], c["sinks"])
            pairs += p
            keys += k
        return {"bytes": keys * c["kv_heads"] * c["dim"] * 2 * es + sum(chunk) * c["heads"] * (4 * c["dim"] + 4)
                + 4 * keys // c["page"], "flops": 4 * pairs * c["heads"] * c["dim"]}
    V, H = c["vocab"], c["hidden"]
    matrix = V * H // 2 + V * H // 32
    if c["op"] == "quantize":  # written, read back, and both bf16 matrices
        return {"bytes": 4 * V * H + 2 * matrix, "flops": 2 * V * H}
    rows = c["batch"] * c["steps"]
    return {"bytes": matrix + rows * H * 2 + rows * V * (2 if c["out"] == "bf16" else 4), "flops": 2 * rows * V * H}


# ---------------------------------------------------------------- prepare --
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 29)
    s = {"rope": _prepare_rope, "attention": _prepare_attention, "quantize": _prepare_quantize,
         "lm_head": _prepare_lm_head}[case["op"]](case, g)
    s["case"] = case
    return s


def _perm(n, g):
    return torch.randperm(n, generator=g, device=DEV)


def _cache_dtype(c):
    return torch.float8_e4m3fn if c["cache"] == "e4m3" else torch.bfloat16


def _frequencies(rot, factor, base=10000.0, trained=4096):
    """Radians a position of each pair, and the factor on cosine and sine: for contexts that are `factor` times the
    trained length, slow pairs divided by it, fast ones kept, a ramp between."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot)
    if factor == 1.0:
        return f, 1.0

    def pair_of(turns):
        return rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), rot - 1)
    ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0


def _prepare_rope(c, g):
    T, Hq, Hk, D, P, NP = c["tokens"] + c["padded"], c["heads"], c["kv_heads"], c["dim"], c["page"], c["pages"]
    # the projection's output: queries, keys and values of a token in one row
    qkv = torch.randn((T, (Hq + 2 * Hk), D), generator=g, device=DEV)
    qkv *= 0.2 + 3.0 * torch.rand((1, Hq + 2 * Hk, 1), generator=g, device=DEV)
    qkv = qkv.to(torch.bfloat16)
    s = {"q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hk], "v": qkv[:, Hq + Hk:], "q_weight": None, "k_weight": None,
         "q_out": torch.zeros((T, Hq, D), device=DEV, dtype=torch.bfloat16)}
    f, s["rope_scale"] = _frequencies(c["rot"], c["factor"])
    s["inv_freq"] = f.to(DEV)
    if c["norm"]:
        for n in ("q_weight", "k_weight"):
            s[n] = (1.0 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16)
    # runs of 8 tokens, as requests have them, anywhere up to the longest context; padding stands at 0
    n8 = -(-c["tokens"] // 8)
    first = torch.randint(0, max(c["far"] - 8, 1), (n8,), generator=g, device=DEV)
    pos = (first[:, None] + torch.arange(8, device=DEV)[None, :]).reshape(-1)[:c["tokens"]]
    s["positions"] = torch.zeros(T, device=DEV, dtype=torch.int64)
    s["positions"][:c["tokens"]] = pos
    if not c["append"]:
        s["k_out"] = torch.zeros((T, Hk, D), device=DEV, dtype=torch.bfloat16)
        return s
    slot = torch.full((T,), -1, device=DEV, dtype=torch.int64)
    base = _perm(NP * P // 8, g)[:n8] * 8
    slot[:c["tokens"]] = (base[:, None] + torch.arange(8, device=DEV)[None, :]).reshape(-1)[:c["tokens"]]
    s["slot_map"], s["k_scale"], s["v_scale"] = slot, None, None
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
    start = torch.tensor([sum(held[:i]) for i in range(B)], device=DEV)
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


def _matrix(V, H, g):
    """A bf16 matrix with rows of unlike sizes, a few large elements and some rows of zeros."""
    w = torch.empty((V, H), device=DEV, dtype=torch.bfloat16).normal_(0.0, 3.0 / math.sqrt(H), generator=g)
    w *= (0.5 + torch.rand((V, 1), generator=g, device=DEV)).to(torch.bfloat16)
    w[:, torch.randint(0, H, (4,), generator=g, device=DEV)] *= 6.0
    w[torch.randint(0, V, (3,), generator=g, device=DEV)] = 0.0
    return w


def _tiles(V, H):
    """Rows and bytes of the library's tiled codes and scales."""
    return (V + 15) // 16, 8 * H, 256 * ((H + 511) // 512)


def _prepare_quantize(c, g):
    V, H = c["vocab"], c["hidden"]
    vt, cb, sb = _tiles(V, H)
    return {"w": _matrix(V, H, g), "tiled": torch.empty((vt, cb), device=DEV, dtype=torch.uint8),
            "scales": torch.empty((vt, sb), device=DEV, dtype=torch.uint8),
            "values": torch.zeros((V, H), device=DEV, dtype=torch.bfloat16)}


def _prepare_lm_head(c, g):
    V, H, rows = c["vocab"], c["hidden"], c["batch"] * c["steps"]
    hidden = torch.randn((rows, H), generator=g, device=DEV)
    hidden[:, torch.randint(0, H, (8,), generator=g, device=DEV)] *= 12.0  # outlier channels
    # a checkpoint in this form: two codes a byte, the even column in the low half, a scale for 32 columns
    codes = torch.randint(0, 256, (V, H // 2), generator=g, device=DEV, dtype=torch.uint8)
    mid = 127 + round(math.log2(0.8 / math.sqrt(H)))
    scales = torch.randint(mid - 2, mid + 2, (V, H // 32), generator=g, device=DEV, dtype=torch.uint8)
    # the order in which the library keeps them: 16 rows by 128 columns, in each four blocks of 32 columns of 16 rows;
    # the scales of four such tiles in a row beside each other
    vt, cb, sb = _tiles(V, H)
    pad = torch.zeros((vt * 16, H // 2), device=DEV, dtype=torch.uint8)
    pad[:V] = codes
    tiled = pad.view(vt, 16, H // 128, 4, 16).permute(0, 2, 3, 1, 4).contiguous().view(vt, cb)
    pad = torch.zeros((vt * 16, sb // 16), device=DEV, dtype=torch.uint8)
    pad[:V, :H // 32] = scales
    order = pad.view(vt, 16, sb // 256, 4, 4).permute(0, 2, 4, 1, 3).contiguous().view(vt, sb)
    dt = torch.bfloat16 if c["out"] == "bf16" else torch.float32
    return {"hidden": hidden.to(torch.bfloat16), "codes": codes, "scales": scales, "tiled": tiled, "tiled_scales": order,
            "out": torch.zeros((c["batch"], c["steps"], V), device=DEV, dtype=dt)}


# -------------------------------------------------------------------- run --
def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "attention": _plain_attention, "quantize": _plain_quantize,
            "lm_head": _plain_lm_head}[state["case"]["op"]](state)


def _run_own(s):
    import markov_draft_sampling_amd as mds
    c = s["case"]
    if c["op"] == "rope":
        if not c["append"]:
            mds.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_out"], s["k_out"],
                             q_weight=s["q_weight"], k_weight=s["k_weight"], interleaved=c["interleaved"],
                             rope_scale=s["rope_scale"])
            return {"q": s["q_out"], "k": s["k_out"]}
        mds.qk_norm_rope_append(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["q_out"], s["k_pages"],
                                s["v_pages"], s["slot_map"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                interleaved=c["interleaved"], rope_scale=s["rope_scale"], k_scale=s["k_scale"],
                                v_scale=s["v_scale"])
        return _append_outputs(s["q_out"], s["k_pages"], s["v_pages"], s)
    if c["op"] == "attention":
        s["workspace"] = mds.paged_attention(
            s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["query_start"], s["seq_lens"], s["out"],
            s["max_q_len"], s["max_seq_len"], window=c["window"], sinks=c["sinks"], k_scale=s["k_scale"],
            v_scale=s["v_scale"], lse=s["lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "quantize":
        mds.quantize_lm_head_mxfp4(s["w"], out=s["tiled"], scales=s["scales"])
        return mds.unpack_lm_head_mxfp4(s["tiled"], s["scales"], out=s["values"])
    mds.lm_head_mxfp4(s["hidden"], s["tiled"], s["tiled_scales"], s["out"], c["steps"])
    return s["out"]


def _append_outputs(q, k, v, s):
    if s["k_scale"] is None:
        return {"q": q, "k_pages": k, "v_pages": v}
    return {"q": q, "k_pages": k.float() * s["k_scale"][:, None], "v_pages": v.float() * s["v_scale"][:, None]}


# ------------------------------------------------------------ plain forms --
def _plain_rope(s):
    c = s["case"]
    R = c["rot"]
    angle = s["positions"].double()[:, None] * s["inv_freq"][None, :]
    cos = (torch.cos(angle) * s["rope_scale"]).float()[:, None, :]
    sin = (torch.sin(angle) * s["rope_scale"]).float()[:, None, :]

    def turn(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + 1e-6) * weight.float()
        a, b = (x[..., 0:R:2], x[..., 1:R:2]) if c["interleaved"] else (x[..., :R // 2], x[..., R // 2:R])
        y, z = a * cos - b * sin, b * cos + a * sin
        y = torch.stack([y, z], dim=-1).flatten(-2) if c["interleaved"] else torch.cat([y, z], dim=-1)
        return torch.cat([y, x[..., R:]], dim=-1)

    q, k = turn(s["q"], s["q_weight"]).to(torch.bfloat16), turn(s["k"], s["k_weight"])
    if not c["append"]:
        return {"q": q, "k": k.to(torch.bfloat16)}
    live = s["slot_map"] >= 0
    # a padding row writes what the first live row's slot gets anyway
    src = torch.where(live, torch.arange(live.numel(), device=live.device), torch.argmax(live.to(torch.int32)))
    slot = s["slot_map"][src]

    def put(x, pages, scale):
        x = x.float()[src]
        new = pages.clone()
        if scale is None:
            new.view(-1, *pages.shape[2:])[slot] = x.to(pages.dtype)
        else:  # codes are put as bytes: indexing knows no 8-bit floating point
            x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(pages.dtype)
            new.view(torch.uint8).view(-1, *pages.shape[2:])[slot] = x.view(torch.uint8)
        return new

    return _append_outputs(q, put(k, s["k_pages"], s["k_scale"]), put(s["v"], s["v_pages"], s["v_scale"]), s)


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
    seen = (key[None, None, :] <= pos[:, :, None]) & (key[None, None, :] < seq[:, None, None])
    seen &= (key[None, None, :] > pos[:, :, None] - c["window"]) | (key < c["sinks"])
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


def _plain_quantize(s):
    V, H = s["w"].shape
    x = s["w"].float().view(V, H // 32, 32)
    amax = x.abs().amax(dim=-1, keepdim=True).clamp(min=2.0 ** -100)
    unit = torch.ldexp(torch.ones_like(amax), torch.frexp(amax).exponent - 3)
    a = (x / unit).abs().clamp(max=6.0)
    # steps of a half below 2, of one below 4, of two above; torch.round goes to the even one
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return (torch.copysign(torch.round(a / step) * step, x) * unit).view(V, H).to(torch.bfloat16)


def _plain_lm_head(s):
    c = s["case"]
    V, H = c["vocab"], c["hidden"]
    half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=s["codes"].device)
    value = torch.cat([half, -half])
    byte = torch.arange(256, device=half.device)
    pair = torch.stack([value[byte % 16], value[byte // 16]], dim=-1)  # both codes of a byte
    w = pair[s["codes"].int()].view(V, H // 32, 32)
    unit = torch.ldexp(torch.ones(s["scales"].shape, device=half.device), s["scales"].int() - 127)
    w = (w * unit[..., None]).view(V, H)
    return (s["hidden"].float() @ w.t()).view(c["batch"], c["steps"], V).to(s["out"].dtype)


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    """The operators' definitions in 64 bits, head by head, request by request and block by block."""
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attention": _exact_attention, "quantize": _exact_quantize,
            "lm_head": _exact_lm_head}[case["op"]](case, s)


def _e4m3_values():
    v = torch.arange(127, dtype=torch.float64)
    e, m = torch.div(v, 8, rounding_mode="floor"), v % 8
    return torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7))


def _nearest(x, values):
    """float64 to the nearest of the values (magnitudes in order), ties to the even place, past the largest to it."""
    val = values.to(x.device)
    top = val.numel() - 1
    a = x.abs().clamp(max=float(val[top]))
    hi = torch.searchsorted(val, a.contiguous()).clamp(max=top)
    lo = (hi - 1).clamp(min=0)
    up, down = val[hi] - a, a - val[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(val[code], x)


def _exact_rope(c, s):
    R, T = c["rot"], s["positions"].numel()
    first = torch.arange(0, R, 2) if c["interleaved"] else torch.arange(R // 2)
    second = first + 1 if c["interleaved"] else first + R // 2
    a = s["positions"].double().view(T, 1) * s["inv_freq"].view(1, -1)
    turn = torch.polar(torch.full_like(a, s["rope_scale"]), a)

    def heads(x, weight):
        out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
        for h in range(x.shape[1]):
            y = x[:, h].double()
            if weight is not None:
                y = y / torch.sqrt(y.pow(2).sum(dim=-1, keepdim=True) / c["dim"] + 1e-6) * weight.double()
            out[:, h] = y
            z = torch.complex(y[:, first].contiguous(), y[:, second].contiguous()) * turn
            out[:, h, first.to(x.device)], out[:, h, second.to(x.device)] = z.real, z.imag
        return out

    q, k = heads(s["q"], s["q_weight"]), heads(s["k"], s["k_weight"])
    if not c["append"]:
        return {"q": q, "k": k}
    out = {"q": q}
    for n, x in (("k", k), ("v", s["v"].double())):
        pages = s[n + "_pages"].float().double()
        flat, x, scale = pages.view(-1, c["kv_heads"], c["dim"]), x[:c["tokens"]], s[n + "_scale"]
        if scale is not None:
            sc = scale.double()[None, :, None]
            flat *= sc
            x = _nearest(x / sc, _e4m3_values()) * sc
        flat[s["slot_map"][:c["tokens"]]] = x
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
        # the places of the keys that some token of the request sees: the first ones, then the window's
        begin = max(0, a + 1 - c["window"])
        key = torch.cat([torch.arange(min(c["sinks"], begin), device=DEV), torch.arange(begin, a + n, device=DEV)])
        slot = s["block_table"][b].long()[key // P] * P + key % P
        for h in range(Hk):
            k, v = (s[x].view(-1, Hk, c["dim"])[:, h].view(torch.uint8 if c["cache"] == "e4m3" else torch.bfloat16)[slot]
                    .view(_cache_dtype(c)).float().double() for x in ("k_pages", "v_pages"))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for i in range(0, n, 512):  # rows in pieces, so that the scores fit
                m = min(512, n - i)
                q = s["q"][t0 + i:t0 + i + m, h * G:(h + 1) * G].double().reshape(m * G, -1)
                x = (q @ k.t()) / math.sqrt(c["dim"])
                at = (a + i + torch.arange(m, device=DEV)).repeat_interleave(G)[:, None]
                x[(key[None, :] > at) | ((key[None, :] + c["window"] <= at) & (key[None, :] >= c["sinks"]))] = -math.inf
                z = torch.logsumexp(x, dim=-1, keepdim=True)
                x -= z
                x.exp_()
                out[t0 + i:t0 + i + m, h * G:(h + 1) * G] = (x @ v).view(m, G, -1)
                lse[t0 + i:t0 + i + m, h * G:(h + 1) * G] = z.view(m, G)
        t0 += n
    return {"out": out, "lse": lse}


def _exact_quantize(c, s):
    V, H = s["w"].shape
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
    out = torch.empty((V, H), dtype=torch.float64, device=DEV)
    for i in range(0, V, 4096):  # rows in pieces: 64 bits are large
        x = s["w"][i:i + 4096].double().view(-1, H // 32, 32)
        amax = x.abs().amax(dim=-1, keepdim=True).clamp(min=2.0 ** -100)
        unit = torch.exp2(torch.floor(torch.log2(amax)) - 2)
        unit = torch.where(unit * 4 > amax, unit / 2, torch.where(unit * 8 <= amax, unit * 2, unit))
        out[i:i + 4096] = (_nearest(x / unit, values) * unit).view(-1, H)
    return out


def _exact_lm_head(c, s):
    V, H = c["vocab"], c["hidden"]
    value = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=DEV) / 2
    z = torch.zeros((c["batch"] * c["steps"], V), dtype=torch.float64, device=DEV)
    for h in range(0, H, 128):  # 128 columns at a time
        code = s["codes"][:, h // 2:h // 2 + 64].int()
        code = torch.stack([code & 15, code >> 4], dim=-1).view(V, 128)
        w = value[code & 7] * (1 - 2 * (code >> 3)).double()
        w = w.view(V, 4, 32) * torch.exp2(s["scales"][:, h // 32:h // 32 + 4].double() - 127.0)[..., None]
        z += s["hidden"][:, h:h + 128].double() @ w.view(V, 128).t()
    return z.view(c["batch"], c["steps"], V)
