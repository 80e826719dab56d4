"""Binding of the serving operators: the paged key/value cache (page tables,
append, attention) and the LM head from an 8-bit matrix. Argument checks and
marshalling only, as in the package's other functions, which re-exports these.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import BF16, E4M3, F32, MdsError, _check, _lib, _need, _ptr

_I32, _I64, _F32, _BF16, _E4M3 = torch.int32, torch.int64, torch.float32, torch.bfloat16, torch.float8_e4m3fn
_vp, _c_sz = ctypes.c_void_p, ctypes.c_size_t


def _call(what, fn, dev, stream, args, tail=()):
    """fn(*args, stream, *tail) on the tensors' device and the given (or that device's current) stream."""
    if stream is None:
        if torch.cuda.current_device() == dev.index:
            rc = fn(*args, _vp(torch.cuda.current_stream(dev).cuda_stream), *tail)
        else:
            with torch.cuda.device(dev):
                rc = fn(*args, _vp(torch.cuda.current_stream(dev).cuda_stream), *tail)
    else:
        _need(stream.device == dev, "the stream belongs to another device than the tensors")
        with torch.cuda.device(dev):
            rc = fn(*args, _vp(stream.cuda_stream), *tail)
    if rc:
        _check(rc, what)


def _workspace(given, nbytes, dev, stream):
    """The caller's workspace, or a new zeroed one made on the stream that the call runs on."""
    if given is not None:
        _need(given.dtype == torch.uint8 and given.is_contiguous() and given.device == dev,
              "workspace must be a contiguous uint8 tensor on the tensors' device")
        return given
    if stream is None:
        return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=dev)
    with torch.cuda.stream(stream):
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=dev)
    return ws


def _vec(t, dtype, n, dev, name):
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous() or t.device != dev:
        raise MdsError(f"{name} must be a contiguous {dtype} tensor of {n} elements on {dev}")


def _opt(t, dtype, n, dev, name):
    if t is not None:
        _vec(t, dtype, n, dev, name)


def _status(t, dev):
    if t is not None:
        _need(t.numel() == 1 and t.element_size() == 4 and t.device == dev, "status: one 4-byte word on the device")


def _pages(k_pages, v_pages, dev):
    """(page size, pages, key heads, head dimension, dtype code) of a pair of page arrays."""
    _need(k_pages.dim() == 4 and v_pages.shape == k_pages.shape and v_pages.dtype == k_pages.dtype,
          "k_pages and v_pages must be [n_pages, page_size, Hkv, D] of one shape and dtype")
    _need(k_pages.device == dev and v_pages.device == dev, "the pages must be on the tensors' device")
    _need(k_pages.stride(3) == 1 and v_pages.stride(3) == 1, "pages must have a unit last stride")
    if k_pages.dtype == _BF16:
        code = BF16
    elif k_pages.dtype == _E4M3:
        code = E4M3
    else:
        raise MdsError(f"unsupported cache dtype {k_pages.dtype}")
    n, p, h, d = k_pages.shape
    return p, n, h, d, code


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
    dev = kv_len.device
    _need(kv_len.is_cuda, "tensors must be on the GPU")
    B, N = chunk_len.numel(), kv_len.numel()
    _need(block_table.dim() == 2 and block_table.shape[0] == N, "block_table must be [n_slots, max_pages]")
    MP, T, NP = block_table.shape[1], slot_map.numel(), free_list.numel()
    for t, dt, n, name in ((kv_len, _I32, N, "kv_len"), (chunk_len, _I32, B, "chunk_len"),
                           (block_table, _I32, N * MP, "block_table"), (pages_held, _I32, N, "pages_held"),
                           (free_list, _I32, NP, "free_list"), (free_count, _I32, 1, "free_count"),
                           (query_start, _I32, B + 1, "query_start"), (seq_lens, _I32, B, "seq_lens"),
                           (positions, _I64, T, "positions"), (slot_map, _I64, T, "slot_map"),
                           (kv_len_out, _I32, N, "kv_len_out"), (pages_held_out, _I32, N, "pages_held_out"),
                           (free_count_out, _I32, 1, "free_count_out")):
        _vec(t, dt, n, dev, name)
    _opt(idx_map, _I32, B, dev, "idx_map")
    _opt(advance, _I32, B, dev, "advance")
    _status(status, dev)
    _call("kv_page_tables", _lib().mds_kv_page_tables, dev, stream,
          (B, N, MP, page_size, NP, T, _ptr(idx_map), _ptr(kv_len), _ptr(advance), advance_add, _ptr(chunk_len),
           _ptr(block_table), _ptr(pages_held), _ptr(free_list), _ptr(free_count), _ptr(query_start), _ptr(seq_lens),
           _ptr(positions), _ptr(slot_map), _ptr(kv_len_out), _ptr(pages_held_out), _ptr(free_count_out),
           _ptr(status)))


def kv_append(k, v, k_pages, v_pages, slot_map, k_scale=None, v_scale=None, status=None, stream=None) -> None:
    """Write the keys and values of new tokens into the cache (mds_kv_append).

    k, v bf16 [T, Hkv, D] (unit last stride); k_pages, v_pages bf16 or
    float8_e4m3fn [n_pages, page_size, Hkv, D] (unit last stride); slot_map
    int64 [T] (< 0 skips the row); k_scale, v_scale float32 [Hkv], needed for
    an 8-bit cache; status: one 4-byte device word or None.
    """
    dev = k.device
    _need(k.is_cuda, "tensors must be on the GPU")
    P, NP, H, D, code = _pages(k_pages, v_pages, dev)
    T = slot_map.numel()
    _need(k.dtype == _BF16 and v.dtype == _BF16 and k.dim() == 3 and k.shape == v.shape and v.device == dev
          and tuple(k.shape) == (T, H, D), "k and v must be bf16 [T, Hkv, D] on one device")
    _need(T == 0 or (k.stride(2) == 1 and v.stride(2) == 1), "k and v must have a unit last stride")
    _vec(slot_map, _I64, T, dev, "slot_map")
    _opt(k_scale, _F32, H, dev, "k_scale")
    _opt(v_scale, _F32, H, dev, "v_scale")
    _status(status, dev)
    ks, vs, kp, vp = k.stride(), v.stride(), k_pages.stride(), v_pages.stride()
    _call("kv_append", _lib().mds_kv_append, dev, stream,
          (T, H, D, _ptr(k), ks[0], ks[1], _ptr(v), vs[0], vs[1], _ptr(k_pages), _ptr(v_pages), code, P, NP, kp[0],
           kp[1], kp[2], vp[0], vp[1], vp[2], _ptr(slot_map), _ptr(k_scale), _ptr(v_scale), _ptr(status)))


def paged_attention_workspace_bytes(T, B, Hq, Hkv, D, max_q_len, max_seq_len, window=0) -> int:
    out = _c_sz()
    _check(_lib().mds_paged_attention_workspace_bytes(T, B, Hq, Hkv, D, max_q_len, max_seq_len, window,
                                                      ctypes.byref(out)), "paged_attention_workspace_bytes")
    return out.value


def paged_attention(q, k_pages, v_pages, block_table, query_start, seq_lens, out, max_q_len, max_seq_len, scale=None,
                    causal=True, window=0, idx_map=None, k_scale=None, v_scale=None, lse=None, workspace=None,
                    stream=None):
    """Attention of every request's new tokens over its paged cache (mds_paged_attention).

    q, out bf16 [T, Hq, D] (unit last stride; D 64 or 128); the cache as for
    kv_append; block_table int32 [n_slots, max_pages]; query_start int32
    [B+1], seq_lens int32 [B]; idx_map int32 [B] or None; max_q_len bounds
    every request's new tokens, max_seq_len guesses the longest sequence;
    scale defaults to 1/sqrt(D); lse float32 [T, Hq] or None. Returns the
    workspace used.
    """
    dev = q.device
    _need(q.is_cuda, "tensors must be on the GPU")
    P, NP, Hk, D, code = _pages(k_pages, v_pages, dev)
    _need(q.dtype == _BF16 and out.dtype == _BF16 and q.dim() == 3 and out.shape == q.shape and q.shape[2] == D
          and out.device == dev, "q and out must be bf16 [T, Hq, D] on one device")
    T, Hq, _ = q.shape
    _need(T == 0 or (q.stride(2) == 1 and out.stride(2) == 1), "q and out must have a unit last stride")
    B = seq_lens.numel()
    _need(block_table.dim() == 2, "block_table must be [n_slots, max_pages]")
    N, MP = block_table.shape
    _vec(block_table, _I32, N * MP, dev, "block_table")
    _vec(query_start, _I32, B + 1, dev, "query_start")
    _vec(seq_lens, _I32, B, dev, "seq_lens")
    _opt(idx_map, _I32, B, dev, "idx_map")
    _opt(k_scale, _F32, Hk, dev, "k_scale")
    _opt(v_scale, _F32, Hk, dev, "v_scale")
    _opt(lse, _F32, T * Hq, dev, "lse")
    if workspace is None:
        workspace = _workspace(None, paged_attention_workspace_bytes(T, B, Hq, Hk, D, max_q_len, max_seq_len, window),
                               dev, stream)
    else:
        _workspace(workspace, 0, dev, stream)
    qs, os, kp, vp = q.stride(), out.stride(), k_pages.stride(), v_pages.stride()
    _call("paged_attention", _lib().mds_paged_attention, dev, stream,
          (T, B, Hq, Hk, D, _ptr(q), qs[0], qs[1], _ptr(k_pages), _ptr(v_pages), code, P, NP, kp[0], kp[1], kp[2],
           vp[0], vp[1], vp[2], _ptr(block_table), N, MP, _ptr(idx_map), _ptr(query_start), _ptr(seq_lens), max_q_len,
           max_seq_len, 1.0 / math.sqrt(D) if scale is None else scale, 1 if causal else 0, window, _ptr(k_scale),
           _ptr(v_scale), _ptr(out), os[0], os[1], _ptr(lse), _ptr(workspace), workspace.numel()))
    return workspace


def lm_head_fp8_tiled_bytes(V, H) -> int:
    out = _c_sz()
    _check(_lib().mds_lm_head_fp8_tiled_bytes(V, H, ctypes.byref(out)), "lm_head_fp8_tiled_bytes")
    return out.value


def _tiled_out(out, V, H, dev):
    shape = ((V + 15) // 16, 16 * H)
    n = lm_head_fp8_tiled_bytes(V, H)
    if out is None:
        out = torch.empty(shape, dtype=_E4M3, device=dev)
    _need(out.dtype == _E4M3 and tuple(out.shape) == shape and out.is_contiguous() and out.device == dev,
          "the tiled matrix must be contiguous float8_e4m3fn [ceil(V/16), 16 H]")
    return out, n


def tile_lm_head_fp8(codes, out=None, stream=None):
    """codes float8_e4m3fn [V, H] (a matrix that has block scales already) in
    the tiled order of mds_tile_lm_head_fp8, [ceil(V/16), 16 H]; returns it."""
    _need(codes.is_cuda and codes.dtype == _E4M3 and codes.dim() == 2 and codes.is_contiguous(),
          "codes must be a contiguous float8_e4m3fn [V, H] GPU tensor")
    V, H = codes.shape
    out, n = _tiled_out(out, V, H, codes.device)
    _call("tile_lm_head_fp8", _lib().mds_tile_lm_head_fp8, codes.device, stream, (V, H, _ptr(codes), _ptr(out), n))
    return out


def quantize_lm_head_fp8(lm_head, out=None, scales=None, stream=None):
    """bf16 [V, H] -> (tiled float8_e4m3fn [ceil(V/16), 16 H], scales float32
    [ceil(V/128), H/128]) by 128 x 128 blocks (mds_quantize_lm_head_fp8)."""
    _need(lm_head.is_cuda and lm_head.dtype == _BF16 and lm_head.dim() == 2 and lm_head.is_contiguous(),
          "lm_head must be a contiguous bf16 [V, H] GPU tensor")
    V, H = lm_head.shape
    dev = lm_head.device
    out, n = _tiled_out(out, V, H, dev)
    blocks = ((V + 127) // 128, H // 128)
    if scales is None:
        scales = torch.empty(blocks, dtype=_F32, device=dev)
    _vec(scales, _F32, blocks[0] * blocks[1], dev, "scales")
    _call("quantize_lm_head_fp8", _lib().mds_quantize_lm_head_fp8, dev, stream,
          (V, H, _ptr(lm_head), _ptr(out), n, _ptr(scales)))
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
    dev = hidden.device
    _need(hidden.is_cuda and hidden.dtype == _BF16 and hidden.dim() == 2 and hidden.stride(1) == 1 and K >= 1
          and hidden.shape[0] % K == 0, "hidden must be bf16 [B*K, H] with unit column stride")
    B, H = hidden.shape[0] // K, hidden.shape[1]
    _need(out.dim() == 3 and out.shape[0] == B and out.shape[1] >= K and out.stride(2) == 1 and out.device == dev,
          "out must be [B, >=K, V] with unit column stride")
    V = out.shape[2]
    _need(lm_head.dtype == _E4M3 and lm_head.is_contiguous() and lm_head.device == dev
          and tuple(lm_head.shape) == ((V + 15) // 16, 16 * H), "lm_head must be the tiled [ceil(V/16), 16 H]")
    _vec(scales, _F32, ((V + 127) // 128) * (H // 128), dev, "scales")
    if out.dtype == _F32:
        code = F32
    elif out.dtype == _BF16:
        code = BF16
    else:
        raise MdsError(f"unsupported dtype {out.dtype}")
    if workspace is None:
        workspace = _workspace(None, lm_head_fp8_workspace_bytes(B, K, V, H), dev, stream)
    else:
        _workspace(workspace, 0, dev, stream)
    _call("lm_head_fp8", _lib().mds_lm_head_fp8, dev, stream,
          (B, K, V, H, _ptr(hidden), hidden.stride(0), _ptr(lm_head), _ptr(scales), _ptr(out), code, out.stride(0),
           out.stride(1), _ptr(workspace), workspace.numel()))
    return workspace
