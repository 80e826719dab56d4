"""Binding of the serving operators: the paged key/value cache (page tables,
append, attention) and the LM head from an 8-bit matrix. Argument checks and
marshalling only, as in the package's other functions, which re-exports these.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import _SIGS, BF16, E4M3, F32, MdsError, _check, _lib, _need

_I32, _I64, _F32, _BF16, _E4M3 = torch.int32, torch.int64, torch.float32, torch.bfloat16, torch.float8_e4m3fn
_c_sz = ctypes.c_size_t

# These calls take a few microseconds on the GPU at decoding sizes, so the checks here are kept cheap: a device is
# compared by its index, pointers are plain integers (0: NULL), the stream is asked for once, and the arguments of the
# calls of a step go over packed (attention's 39 ctypes arguments cost 3.6 us, packed 0.9).


def _current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def _call(what, fn, index, stream, args):
    """fn(*args, stream) on the tensors' device and the given (or that device's current) stream."""
    if stream is None and torch.cuda.current_device() == index:
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
           for i, name in enumerate(("kv_page_tables", "kv_append", "paged_attention", "lm_head_fp8"))}


def _packed(what, index, stream, args):
    """mds_<what>(*args, stream) by mds_call_packed, as _call."""
    call, layout = _PACKED[what]
    try:
        data = layout.pack(*args)
    except struct.error as e:
        raise MdsError(f"{what}: an argument is no integer or out of range: {e}") from None
    _call(what, _lib().mds_call_packed, index, stream, (call, data, len(args)))


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
    dev = _index(q)
    (NP, P, Hk, D), code, kp, vp = _pages(k_pages, v_pages, dev)
    shape = q.shape
    _need(q.dtype is _BF16 and out.dtype is _BF16 and len(shape) == 3 and out.shape == shape and shape[2] == D
          and out.get_device() == dev, "q and out must be bf16 [T, Hq, D] on one device")
    T, Hq, _ = shape
    qs, os = q.stride(), out.stride()
    _need(T == 0 or (qs[2] == 1 and os[2] == 1), "q and out must have a unit last stride")
    B = seq_lens.numel()
    _need(block_table.dim() == 2, "block_table must be [n_slots, max_pages]")
    N, MP = block_table.shape
    if workspace is None:
        workspace = _new_workspace(paged_attention_workspace_bytes(T, B, Hq, Hk, D, max_q_len, max_seq_len, window),
                                   dev, stream)
    else:
        _check_workspace(workspace, dev)
    _packed("paged_attention", dev, stream,
          (T, B, Hq, Hk, D, q.data_ptr(), qs[0], qs[1], k_pages.data_ptr(), v_pages.data_ptr(), code, P, NP, kp[0], kp[1],
           kp[2], vp[0], vp[1], vp[2], _vec(block_table, _I32, N * MP, dev, "block_table"), N, MP,
           _opt(idx_map, _I32, B, dev, "idx_map"), _vec(query_start, _I32, B + 1, dev, "query_start"),
           _vec(seq_lens, _I32, B, dev, "seq_lens"), max_q_len, max_seq_len, 1.0 / math.sqrt(D) if scale is None else scale,
           1 if causal else 0, window, _opt(k_scale, _F32, Hk, dev, "k_scale"), _opt(v_scale, _F32, Hk, dev, "v_scale"),
           out.data_ptr(), os[0], os[1], _opt(lse, _F32, T * Hq, dev, "lse"), workspace.data_ptr(), workspace.numel()))
    return workspace


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
