"""Binding of the serving operators: the paged key/value cache (page tables,
norm and rotation, append, attention) and the LM heads from 8-bit and 4-bit
matrices. Argument checks and marshalling only, as in the package's other
functions, which re-exports these.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import struct

import torch

from . import _SIGS, BF16, E4M3, F32, MdsError, _check, _lib, _need

_I32, _I64, _F32, _BF16, _E4M3 = torch.int32, torch.int64, torch.float32, torch.bfloat16, torch.float8_e4m3fn
_F64, _U8 = torch.float64, torch.uint8
_c_sz = ctypes.c_size_t

# These calls take a few microseconds on the GPU at decoding sizes, so the checks here are kept cheap: a device is
# compared by its index, pointers are plain integers (0: NULL), the stream is asked for once, and the arguments of the
# calls of a step go over packed (39 ctypes arguments cost 3.6 us, packed 0.9). Those whose checks would
# outlast their kernels all the same are checked and called by _calls, which is compiled; where it is not built, attention
# is called from here (11 to 13 us of host time for one token instead of 8) and the others raise an error that says so.


def _current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)  # (there are tensors on the GPU already)


def _call(what, fn, index, stream, args):
    """fn(*args, stream) on the tensors' device and the given (or that device's current) stream."""
    if stream is None and _current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        if stream is not None and stream.device.index != index:
            raise MdsError("the stream belongs to another device than the tensors")
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, what)


# mds_call_packed's numbers and the arguments' layout: 8 bytes each, floats as doubles
_PACKED = {name: (i, struct.Struct("".join("d" if t is ctypes.c_float else "q" for t in _SIGS["mds_" + name][0][:-1])))
           for i, name in ((0, "kv_page_tables"), (1, "kv_append"), (2, "paged_attention"), (3, "lm_head_fp8"))}


def _packed(what, index, stream, args):
    """mds_<what>(*args, stream) by mds_call_packed, as _call."""
    call, layout = _PACKED[what]
    try:
        data = layout.pack(*args)
    except struct.error as e:
        raise MdsError(f"{what}: an argument is no integer or out of range: {e}") from None
    _call(what, _lib().mds_call_packed, index, stream, (call, data, len(args)))


_CALLS = None  # the module of the compiled calls, once it is loaded; False: there is none for this interpreter


def _calls(needed=True):
    """The module of the compiled calls; None where there is none and it is not needed."""
    global _CALLS
    how = "build them with `python -m markov_draft_sampling_amd.build`"
    if _CALLS is None:
        _lib()
        if importlib.util.find_spec("._calls", __package__) is None:
            _CALLS = False
        else:
            try:
                from . import _calls as m
            except ImportError as e:
                raise MdsError(f"the compiled calls do not load ({e}): {how}") from None
            m.set_error(MdsError)
            _CALLS = m
    if needed and not _CALLS:
        raise MdsError(f"there are no compiled calls for this interpreter: {how}")
    return _CALLS or None


def _compiled(fn, index, stream, *args):
    """fn(*args, stream) of _calls, as _call."""
    if stream is None and _current_device() == index:
        fn(*args, _raw_stream(index))
        return
    if stream is not None and stream.device.index != index:
        raise MdsError("the stream belongs to another device than the tensors")
    with torch.cuda.device(index):
        fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)


def _on(stream, make, *args, **kw):
    """make(*args, **kw) on the stream that a call runs on: memory that its results take over from a freed tensor may
    still be in use on another stream."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _new_workspace(nbytes, index, stream):
    """Memory for a call's partial results, with a cleared status word in front (which is all that has to be)."""
    def make():
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=f"cuda:{index}")
        ws[:256].zero_()
        return ws
    return _on(stream, make)


def _check_workspace(ws, index):
    if ws.dtype is not torch.uint8 or ws.get_device() != index or not ws.is_contiguous():
        raise MdsError("workspace must be a contiguous uint8 tensor on the tensors' device")


def _index(t):
    """The device index of a GPU tensor (the first argument of a call, which the others have to be beside)."""
    i = t.get_device()
    if i < 0:
        raise MdsError("tensors must be on the GPU")
    return i


def _vec(t, dtype, n, index, name):
    """The pointer of a contiguous tensor of n elements on the device."""
    if t.dtype is not dtype or t.numel() != n or t.get_device() != index or not t.is_contiguous():
        raise MdsError(f"{name} must be a contiguous {dtype} tensor of {n} elements on cuda:{index}")
    return t.data_ptr()


def _opt(t, dtype, n, index, name):
    return 0 if t is None else _vec(t, dtype, n, index, name)


def _status(t, index):
    if t is None:
        return 0
    if t.numel() != 1 or t.element_size() != 4 or t.get_device() != index:
        raise MdsError("status: one 4-byte word on the device")
    return t.data_ptr()


def _pages(k_pages, v_pages, index):
    """(shape, dtype code, strides of keys, strides of values) of a pair of page arrays."""
    shape, dtype = k_pages.shape, k_pages.dtype
    if len(shape) != 4 or v_pages.shape != shape or v_pages.dtype is not dtype:
        raise MdsError("k_pages and v_pages must be [n_pages, page_size, Hkv, D] of one shape and dtype")
    if k_pages.get_device() != index or v_pages.get_device() != index:
        raise MdsError("the pages must be on the tensors' device")
    ks, vs = k_pages.stride(), v_pages.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise MdsError("pages must have a unit last stride")
    if dtype is _BF16:
        return shape, BF16, ks, vs
    if dtype is _E4M3:
        return shape, E4M3, ks, vs
    raise MdsError(f"unsupported cache dtype {dtype}")


def kv_page_tables(kv_len, chunk_len, block_table, pages_held, free_list, free_count, page_size, query_start, seq_lens,
                   positions, slot_map, kv_len_out, pages_held_out, free_count_out, status=None, idx_map=None,
                   advance=None, advance_add=0, stream=None) -> None:
    """Pages, positions and slots of the next new tokens (mds_kv_page_tables).

    kv_len, pages_held int32 [n_slots]; chunk_len int32 [B] (< 0 releases the
    request); block_table int32 [n_slots, max_pages]; free_list int32
    [n_pages], free_count int32 [1]; idx_map int32 [B] or None; advance int32
    [B] or None (num_accepted of the last verification, with advance_add=1).
    Writes query_start [B+1], seq_lens [B], positions and slot_map int64
    [max_tokens], the new entries of block_table, the released pages of
    free_list, and kv_len_out, pages_held_out, free_count_out, which may be
    the inputs. status: one 4-byte device word or None.
    """
    dev = _index(kv_len)
    B, N = chunk_len.numel(), kv_len.numel()
    _need(block_table.dim() == 2 and block_table.shape[0] == N, "block_table must be [n_slots, max_pages]")
    MP, T, NP = block_table.shape[1], slot_map.numel(), free_list.numel()
    _packed("kv_page_tables", dev, stream,
          (B, N, MP, page_size, NP, T, _opt(idx_map, _I32, B, dev, "idx_map"), _vec(kv_len, _I32, N, dev, "kv_len"),
           _opt(advance, _I32, B, dev, "advance"), advance_add, _vec(chunk_len, _I32, B, dev, "chunk_len"),
           _vec(block_table, _I32, N * MP, dev, "block_table"), _vec(pages_held, _I32, N, dev, "pages_held"),
           _vec(free_list, _I32, NP, dev, "free_list"), _vec(free_count, _I32, 1, dev, "free_count"),
           _vec(query_start, _I32, B + 1, dev, "query_start"), _vec(seq_lens, _I32, B, dev, "seq_lens"),
           _vec(positions, _I64, T, dev, "positions"), _vec(slot_map, _I64, T, dev, "slot_map"),
           _vec(kv_len_out, _I32, N, dev, "kv_len_out"), _vec(pages_held_out, _I32, N, dev, "pages_held_out"),
           _vec(free_count_out, _I32, 1, dev, "free_count_out"), _status(status, dev)))


def kv_append(k, v, k_pages, v_pages, slot_map, k_scale=None, v_scale=None, status=None, stream=None) -> None:
    """Write the keys and values of new tokens into the cache (mds_kv_append).

    k, v bf16 [T, Hkv, D] (unit last stride); k_pages, v_pages bf16 or
    float8_e4m3fn [n_pages, page_size, Hkv, D] (unit last stride); slot_map
    int64 [T] (< 0 skips the row); k_scale, v_scale float32 [Hkv], needed for
    an 8-bit cache; status: one 4-byte device word or None.
    """
    dev = _index(k)
    (NP, P, H, D), code, kp, vp = _pages(k_pages, v_pages, dev)
    T = slot_map.numel()
    _need(k.dtype is _BF16 and v.dtype is _BF16 and k.shape == v.shape and k.shape == (T, H, D)
          and v.get_device() == dev, "k and v must be bf16 [T, Hkv, D] on one device")
    ks, vs = k.stride(), v.stride()
    _need(T == 0 or (ks[2] == 1 and vs[2] == 1), "k and v must have a unit last stride")
    _packed("kv_append", dev, stream,
          (T, H, D, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], k_pages.data_ptr(), v_pages.data_ptr(), code,
           P, NP, kp[0], kp[1], kp[2], vp[0], vp[1], vp[2], _vec(slot_map, _I64, T, dev, "slot_map"),
           _opt(k_scale, _F32, H, dev, "k_scale"), _opt(v_scale, _F32, H, dev, "v_scale"), _status(status, dev)))


def rope_frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, trained_len=0, beta_fast=32.0, beta_slow=1.0,
                     device="cuda"):
    """(inv_freq float64 [rotary_dim / 2] in radians a position, rope_scale) for qk_norm_rope.

    Pair i turns by base^(-2 i / rotary_dim) a position. scaling, for contexts
    factor times as long as those trained on: "linear" divides every frequency
    by factor; "ntk" takes base * factor^(rotary_dim / (rotary_dim - 2)), which
    divides the slowest one by it and keeps the fastest; "yarn" (Peng et al.,
    "YaRN", 2023) divides the pairs that turn less than beta_slow times within
    trained_len positions, keeps those of more than beta_fast, goes over in a
    ramp between, and gives rope_scale = 0.1 ln(factor) + 1 (1 for the others).
    """
    _need(rotary_dim >= 2 and rotary_dim % 2 == 0 and base > 1.0, "rotary_dim must be even, base above 1")
    _need(factor >= 1.0, "factor must be at least 1")
    i = torch.arange(rotary_dim // 2, dtype=_F64)
    if scaling == "ntk":
        _need(rotary_dim > 2, "ntk scaling needs more than one pair")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f, rope_scale = base ** (-2.0 * i / rotary_dim), 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        _need(trained_len >= 1 and beta_fast > beta_slow > 0, "yarn scaling needs trained_len and beta_fast > beta_slow > 0")
        lo, hi = (rotary_dim * math.log(trained_len / (turns * 2 * math.pi)) / (2 * math.log(base))
                  for turns in (beta_fast, beta_slow))
        if hi <= 0:  # even the fastest pair turns beta_slow times at most
            ramp = torch.ones_like(i)
        else:
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rotary_dim - 1)
            ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f, rope_scale = f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "ntk"):
        raise MdsError(f"unknown scaling {scaling!r}")
    return f.to(device), rope_scale


def qk_norm_rope(q, k, positions, inv_freq, q_out, k_out, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                 rope_scale=1.0, stream=None) -> None:
    """Norm and rotation of queries and keys, head by head (mds_qk_norm_rope).

    q, q_out bf16 [T, Hq, D], k, k_out bf16 [T, Hkv, D] (unit last stride; an
    output may be its input); positions int64 [T]; inv_freq float64 [R / 2]
    for the first R columns of a head, or None (no rotation); q_weight,
    k_weight bf16 [D] or None (no norm); interleaved pairs columns (2 i, 2 i +
    1) instead of (i, i + R / 2); rope_scale multiplies cosine and sine.
    """
    _compiled(_calls().qk_norm_rope, _index(q), stream, q, k, positions, inv_freq, q_out, k_out, q_weight, k_weight, eps,
              interleaved, rope_scale)


def qk_norm_rope_append(q, k, v, positions, inv_freq, q_out, k_pages, v_pages, slot_map, q_weight=None, k_weight=None,
                        eps=1e-6, interleaved=False, rope_scale=1.0, k_scale=None, v_scale=None, status=None,
                        stream=None) -> None:
    """qk_norm_rope with the keys, and the values v beside them, written into
    the cache (mds_qk_norm_rope_append).

    q, k, positions to rope_scale as for qk_norm_rope; v bf16 [T, Hkv, D]; the
    pages, slot_map, scales and status as for kv_append.
    """
    _compiled(_calls().qk_norm_rope_append, _index(q), stream, q, k, v, positions, inv_freq, q_out, k_pages, v_pages,
              slot_map, q_weight, k_weight, eps, interleaved, rope_scale, k_scale, v_scale, status)


def paged_attention_workspace_bytes(T, B, Hq, Hkv, D, max_q_len, max_seq_len, window=0, sinks=0) -> int:
    out = _c_sz()
    _check(_lib().mds_paged_attention_sinks_workspace_bytes(T, B, Hq, Hkv, D, max_q_len, max_seq_len, window, sinks,
                                                            ctypes.byref(out)), "paged_attention_workspace_bytes")
    return out.value


def paged_attention(q, k_pages, v_pages, block_table, query_start, seq_lens, out, max_q_len, max_seq_len, scale=None,
                    causal=True, window=0, idx_map=None, k_scale=None, v_scale=None, lse=None, workspace=None,
                    stream=None, sinks=0):
    """Attention of every request's new tokens over its paged cache (mds_paged_attention, mds_paged_attention_sinks).

    q, out bf16 [T, Hq, D] (unit last stride; D 64 or 128); the cache as for
    kv_append; block_table int32 [n_slots, max_pages]; query_start int32
    [B+1], seq_lens int32 [B]; idx_map int32 [B] or None; max_q_len bounds
    every request's new tokens, max_seq_len guesses the longest sequence;
    scale defaults to 1/sqrt(D); window bounds how far back a token sees, but for
    the first sinks tokens; lse float32 [T, Hq] or None. Returns the workspace used.
    """
    dev = _index(q)
    if workspace is None:
        _need(q.dim() == 3 and k_pages.dim() == 4, "q must be [T, Hq, D], the pages [n_pages, page_size, Hkv, D]")
        T, Hq, D = q.shape
        nbytes = paged_attention_workspace_bytes(T, seq_lens.numel(), Hq, k_pages.shape[2], D, max_q_len, max_seq_len,
                                                 window, sinks)
        workspace = _new_workspace(nbytes, dev, stream)
    args = (q, k_pages, v_pages, block_table, query_start, seq_lens, out, max_q_len, max_seq_len, scale, causal, window,
            sinks, idx_map, k_scale, v_scale, lse, workspace)
    calls = _calls(needed=False)
    if calls is None:
        _attention(dev, stream, *args)
    else:
        _compiled(calls.paged_attention, dev, stream, *args)
    return workspace


def _heads(t, shape, index, name):
    """(pointer, token stride, head stride) of bf16 [T, H, D] with a unit last stride."""
    st = t.stride()
    if t.dtype is not _BF16 or t.shape != shape or t.get_device() != index or (st[2] != 1 and t.numel()):
        raise MdsError(f"{name} must be bf16 {list(shape)} with a unit last stride on cuda:{index}")
    return t.data_ptr(), st[0], st[1]


def _attention(dev, stream, q, k_pages, v_pages, block_table, query_start, seq_lens, out, max_q_len, max_seq_len, scale,
               causal, window, sinks, idx_map, k_scale, v_scale, lse, workspace):
    """_calls' paged_attention, in Python."""
    (NP, P, Hk, D), code, kp, vp = _pages(k_pages, v_pages, dev)
    _need(q.dim() == 3, "q must be bf16 [T, Hq, D]")
    T, Hq, _ = q.shape
    B = seq_lens.numel()
    _need(block_table.dim() == 2, "block_table must be [n_slots, max_pages]")
    N, MP = block_table.shape
    _check_workspace(workspace, dev)
    args = (T, B, Hq, Hk, D, *_heads(q, (T, Hq, D), dev, "q"), k_pages.data_ptr(), v_pages.data_ptr(), code, P, NP, *kp[:3],
            *vp[:3], _vec(block_table, _I32, N * MP, dev, "block_table"), N, MP, _opt(idx_map, _I32, B, dev, "idx_map"),
            _vec(query_start, _I32, B + 1, dev, "query_start"), _vec(seq_lens, _I32, B, dev, "seq_lens"), max_q_len,
            max_seq_len, 1.0 / math.sqrt(D) if scale is None else scale, 1 if causal else 0,
            *((window, sinks) if sinks else (window,)),
            _opt(k_scale, _F32, Hk, dev, "k_scale"), _opt(v_scale, _F32, Hk, dev, "v_scale"),
            *_heads(out, (T, Hq, D), dev, "out"), _opt(lse, _F32, T * Hq, dev, "lse"), workspace.data_ptr(), workspace.numel())
    if not sinks:
        _packed("paged_attention", dev, stream, args)
        return
    try:
        _ATTENTION.pack(*args)  # (ctypes would cut integers to their types' size)
    except struct.error as e:
        raise MdsError(f"paged_attention: an argument is no integer or out of range: {e}") from None
    _call("paged_attention", _lib().mds_paged_attention_sinks, dev, stream, args)


# the types and ranges of mds_paged_attention_sinks' arguments
_ATTENTION = struct.Struct("=" + "".join({ctypes.c_int: "i", ctypes.c_int64: "q", ctypes.c_float: "d"}.get(t, "Q")
                                         for t in _SIGS["mds_paged_attention_sinks"][0][:-1]))


def lm_head_fp8_tiled_bytes(V, H) -> int:
    out = _c_sz()
    _check(_lib().mds_lm_head_fp8_tiled_bytes(V, H, ctypes.byref(out)), "lm_head_fp8_tiled_bytes")
    return out.value


def _tiled_out(out, V, H, dev, stream):  # dev: the device's index
    shape = ((V + 15) // 16, 16 * H)
    n = lm_head_fp8_tiled_bytes(V, H)
    if out is None:
        out = _on(stream, torch.empty, shape, dtype=_E4M3, device=f"cuda:{dev}")
    _need(out.dtype is _E4M3 and out.shape == shape and out.is_contiguous() and out.get_device() == dev,
          "the tiled matrix must be contiguous float8_e4m3fn [ceil(V/16), 16 H]")
    return out, n


def tile_lm_head_fp8(codes, out=None, stream=None):
    """codes float8_e4m3fn [V, H] (a matrix that has block scales already) in
    the tiled order of mds_tile_lm_head_fp8, [ceil(V/16), 16 H]; returns it."""
    _need(codes.is_cuda and codes.dtype == _E4M3 and codes.dim() == 2 and codes.is_contiguous(),
          "codes must be a contiguous float8_e4m3fn [V, H] GPU tensor")
    V, H = codes.shape
    dev = _index(codes)
    out, n = _tiled_out(out, V, H, dev, stream)
    _call("tile_lm_head_fp8", _lib().mds_tile_lm_head_fp8, dev, stream, (V, H, codes.data_ptr(), out.data_ptr(), n))
    return out


def quantize_lm_head_fp8(lm_head, out=None, scales=None, stream=None):
    """bf16 [V, H] -> (tiled float8_e4m3fn [ceil(V/16), 16 H], scales float32
    [ceil(V/128), H/128]) by 128 x 128 blocks (mds_quantize_lm_head_fp8)."""
    _need(lm_head.is_cuda and lm_head.dtype == _BF16 and lm_head.dim() == 2 and lm_head.is_contiguous(),
          "lm_head must be a contiguous bf16 [V, H] GPU tensor")
    V, H = lm_head.shape
    dev = _index(lm_head)
    out, n = _tiled_out(out, V, H, dev, stream)
    blocks = ((V + 127) // 128, H // 128)
    if scales is None:
        scales = _on(stream, torch.empty, blocks, dtype=_F32, device=f"cuda:{dev}")
    _call("quantize_lm_head_fp8", _lib().mds_quantize_lm_head_fp8, dev, stream,
          (V, H, lm_head.data_ptr(), out.data_ptr(), n, _vec(scales, _F32, blocks[0] * blocks[1], dev, "scales")))
    return out, scales


def lm_head_fp8_workspace_bytes(B, K, V, H) -> int:
    out = _c_sz()
    _check(_lib().mds_lm_head_fp8_workspace_bytes(B, K, V, H, ctypes.byref(out)), "lm_head_fp8_workspace_bytes")
    return out.value


def lm_head_fp8(hidden, lm_head, scales, out, K, workspace=None, stream=None):
    """Logits from an 8-bit LM head (mds_lm_head_fp8).

    hidden bf16 [B*K, H] (row b*K + k, unit column stride); lm_head and scales
    from tile_lm_head_fp8 / quantize_lm_head_fp8; out float32 or bf16
    [B, >=K, V] with unit column stride (rows k < K are written). Returns the
    workspace used.
    """
    dev = _index(hidden)
    _need(hidden.dtype is _BF16 and hidden.dim() == 2 and hidden.stride(1) == 1 and K >= 1 and hidden.shape[0] % K == 0,
          "hidden must be bf16 [B*K, H] with unit column stride")
    rows, H = hidden.shape
    B = rows // K
    _need(out.dim() == 3 and out.shape[0] == B and out.shape[1] >= K and out.stride(2) == 1 and out.get_device() == dev,
          "out must be [B, >=K, V] with unit column stride")
    V = out.shape[2]
    _need(lm_head.dtype is _E4M3 and lm_head.is_contiguous() and lm_head.get_device() == dev
          and lm_head.shape == ((V + 15) // 16, 16 * H), "lm_head must be the tiled [ceil(V/16), 16 H]")
    if out.dtype is _F32:
        code = F32
    elif out.dtype is _BF16:
        code = BF16
    else:
        raise MdsError(f"unsupported dtype {out.dtype}")
    if workspace is None:
        workspace = _new_workspace(lm_head_fp8_workspace_bytes(B, K, V, H), dev, stream)
    else:
        _check_workspace(workspace, dev)
    _packed("lm_head_fp8", dev, stream,
          (B, K, V, H, hidden.data_ptr(), hidden.stride(0), lm_head.data_ptr(),
           _vec(scales, _F32, ((V + 127) // 128) * (H // 128), dev, "scales"), out.data_ptr(), code, out.stride(0),
           out.stride(1), workspace.data_ptr(), workspace.numel()))
    return workspace


_CODES = tuple(getattr(torch, n) for n in ("uint8", "float4_e2m1fn_x2") if hasattr(torch, n))
_SCALES = tuple(getattr(torch, n) for n in ("uint8", "float8_e8m0fnu") if hasattr(torch, n))


def lm_head_mxfp4_bytes(V, H):
    """(bytes of the tiled codes, of the tiled scales) of a 4-bit matrix [V, H]."""
    codes, scales = _c_sz(), _c_sz()
    _check(_lib().mds_lm_head_mxfp4_bytes(V, H, ctypes.byref(codes), ctypes.byref(scales)), "lm_head_mxfp4_bytes")
    return codes.value, scales.value


def _mx_shapes(V, H):
    return ((V + 15) // 16, 8 * H), ((V + 15) // 16, 256 * ((H + 511) // 512))


def _mx_tiles(lm_head, scales, V, H, dev):
    """The tiled codes and scales of a matrix [V, H], checked."""
    cs, ss = _mx_shapes(V, H)
    _need(lm_head.dtype is _U8 and lm_head.shape == cs and lm_head.is_contiguous() and lm_head.get_device() == dev,
          "the tiled codes must be contiguous uint8 [ceil(V/16), 8 H]")
    _need(scales.dtype is _U8 and scales.shape == ss and scales.is_contiguous() and scales.get_device() == dev,
          "the tiled scales must be contiguous uint8 [ceil(V/16), 256 ceil(H/512)]")


def _mx_out(out, scales, V, H, dev, stream):
    codes, scale_bytes = lm_head_mxfp4_bytes(V, H)
    cs, ss = _mx_shapes(V, H)
    if out is None:
        out = _on(stream, torch.empty, cs, dtype=_U8, device=f"cuda:{dev}")
    if scales is None:
        scales = _on(stream, torch.empty, ss, dtype=_U8, device=f"cuda:{dev}")
    _mx_tiles(out, scales, V, H, dev)
    return out, codes, scales, scale_bytes


def tile_lm_head_mxfp4(codes, scales, out=None, out_scales=None, stream=None):
    """Codes uint8 (or float4_e2m1fn_x2) [V, H/2] and scales uint8 (or
    float8_e8m0fnu) [V, H/32] (a matrix that is in 4 bits already) in the tiled
    order of mds_tile_lm_head_mxfp4: (uint8 [ceil(V/16), 8 H], uint8
    [ceil(V/16), 256 ceil(H/512)])."""
    _need(codes.is_cuda and codes.dtype in _CODES and codes.dim() == 2 and codes.is_contiguous(),
          "codes must be a contiguous uint8 [V, H/2] GPU tensor")
    dev = _index(codes)
    V, H = codes.shape[0], 2 * codes.shape[1]
    _need(scales.dtype in _SCALES and scales.shape == (V, H // 32) and scales.is_contiguous()
          and scales.get_device() == dev, "scales must be a contiguous uint8 [V, H/32] beside the codes")
    out, n, out_scales, m = _mx_out(out, out_scales, V, H, dev, stream)
    _call("tile_lm_head_mxfp4", _lib().mds_tile_lm_head_mxfp4, dev, stream,
          (V, H, codes.data_ptr(), scales.data_ptr(), out.data_ptr(), n, out_scales.data_ptr(), m))
    return out, out_scales


def quantize_lm_head_mxfp4(lm_head, out=None, scales=None, stream=None):
    """bf16 [V, H] -> (tiled codes, tiled scales) of tile_lm_head_mxfp4, a scale
    for 32 columns of a row (mds_quantize_lm_head_mxfp4)."""
    _need(lm_head.is_cuda and lm_head.dtype is _BF16 and lm_head.dim() == 2 and lm_head.is_contiguous(),
          "lm_head must be a contiguous bf16 [V, H] GPU tensor")
    V, H = lm_head.shape
    dev = _index(lm_head)
    out, n, scales, m = _mx_out(out, scales, V, H, dev, stream)
    _call("quantize_lm_head_mxfp4", _lib().mds_quantize_lm_head_mxfp4, dev, stream,
          (V, H, lm_head.data_ptr(), out.data_ptr(), n, scales.data_ptr(), m))
    return out, scales


def unpack_lm_head_mxfp4(lm_head, scales, V=None, out=None, stream=None):
    """The weights of a tiled 4-bit matrix in bf16 [V, H], which holds them
    exactly; V rows of it, out's or all."""
    dev = _index(lm_head)
    _need(lm_head.dim() == 2 and lm_head.shape[1] % 8 == 0, "the tiled codes must be [ceil(V/16), 8 H]")
    H = lm_head.shape[1] // 8
    if V is None:
        V = 16 * lm_head.shape[0] if out is None else out.shape[0]
    _mx_tiles(lm_head, scales, V, H, dev)
    if out is None:
        out = _on(stream, torch.empty, (V, H), dtype=_BF16, device=f"cuda:{dev}")
    _need(out.dtype is _BF16 and out.shape == (V, H) and out.is_contiguous() and out.get_device() == dev,
          "out must be a contiguous bf16 [V, H]")
    _call("unpack_lm_head_mxfp4", _lib().mds_unpack_lm_head_mxfp4, dev, stream,
          (V, H, lm_head.data_ptr(), scales.data_ptr(), out.data_ptr()))
    return out


def lm_head_mxfp4(hidden, lm_head, scales, out, K, stream=None) -> None:
    """Logits from a 4-bit LM head (mds_lm_head_mxfp4).

    hidden bf16 [B*K, H] (row b*K + k, unit column stride); lm_head and scales
    from tile_lm_head_mxfp4 / quantize_lm_head_mxfp4; out float32 or bf16
    [B, >=K, V] with unit column stride (rows k < K are written).
    """
    _compiled(_calls().lm_head_mxfp4, _index(hidden), stream, hidden, lm_head, scales, out, K)
