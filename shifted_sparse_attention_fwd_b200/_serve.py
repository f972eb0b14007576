"""Binding of the serving entries of libs2attn.so: rotation and append, and decode over a paged
key/value cache (include/s2attn.h, "Serving").

Argument marshalling only, as in _lib.py. A decoding step is a few microseconds of GPU work, so
these functions keep their own cost low: one pass over the arguments and one ctypes call. Tensors
that belong to another device than the current one are run on that device's current stream.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from ._lib import S2ATTN_OK, S2AttnError, _stream, lib

_BF16, _I32 = torch.bfloat16, torch.int32


def _on(stream, device):
    """What is allocated for a call belongs to the stream that the call runs on."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _run(name, device, stream, call):
    """call(stream handle) with `device` current; raises on a failed status."""
    if device.index == torch.cuda.current_device():
        status = call(_stream(stream))
    else:
        with torch.cuda.device(device):
            status = call(_stream(stream))
    if status != S2ATTN_OK:
        raise S2AttnError(status, name)


def _rows(t, name, shape, device):
    """Row stride of a bf16 [rows, heads, d] tensor whose (heads, d) block is contiguous."""
    if t.dtype != _BF16:
        raise ValueError(f"{name}: expected bf16, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name}: expected a tensor on {device}, got {t.device}")
    st = t.stride()
    if st[2] != 1 or st[1] != shape[2]:
        raise ValueError(f"{name}: expected contiguous (heads, d) blocks")
    return st[0]


def _cache_strides(t, name, shape, device):
    """(page, token) strides of a bf16 [pages, page_size, Hkv, d] cache."""
    if t.dtype != _BF16:
        raise ValueError(f"{name}: expected bf16, got {t.dtype}")
    if t.dim() != 4 or t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name}: expected a tensor on {device}, got {t.device}")
    st = t.stride()
    if st[3] != 1 or st[2] != shape[3]:
        raise ValueError(f"{name}: expected contiguous (Hkv, d) blocks")
    return st[0], st[1]


def _ints(t, name, shape, device):
    if t.dtype != _I32 or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous int32 tensor of shape {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def s2attn_rope_append(q, q_rot, k, k_rot, v, k_cache, v_cache, block_table, cache_lens,
                       cu_seqlens=None, base=10000.0, pi_scale=1.0, stream=None):
    """Turn the new tokens' q [T,Hq,d] into q_rot (both may be None; q_rot may be q) and k [T,Hkv,d]
    into the paged cache (and k_rot unless None; may be k), and copy v [T,Hkv,d] into the cache.
    k_cache, v_cache [pages,page_size,Hkv,d]; block_table int32 [B,max_pages]; cache_lens int32 [B],
    the tokens of each sequence including the new ones; cu_seqlens int32 [B+1], the sequences' first
    rows, or None for one new token per sequence. All but the strides is checked in include/s2attn.h's
    terms; a bad page or length on the device is reported by s2attn_get_device_error."""
    dev = k.device
    T, Hkv, d = k.shape
    pages, page_size = k_cache.shape[:2]
    B, max_pages = block_table.shape
    Hq, q_st, qr_st = Hkv, Hkv * d, Hkv * d
    if (q is None) != (q_rot is None):
        raise ValueError("q and q_rot go together")
    if q is not None:
        Hq = q.shape[1]
        q_st, qr_st = _rows(q, "q", (T, Hq, d), dev), _rows(q_rot, "q_rot", (T, Hq, d), dev)
    k_st, v_st = _rows(k, "k", k.shape, dev), _rows(v, "v", k.shape, dev)
    kr_st = k_st if k_rot is None else _rows(k_rot, "k_rot", k.shape, dev)
    cache = (pages, page_size, Hkv, d)
    strides = (ctypes.c_longlong * 9)(
        q_st, qr_st, k_st, kr_st, v_st, *_cache_strides(k_cache, "k_cache", cache, dev),
        *_cache_strides(v_cache, "v_cache", cache, dev))
    table = _ints(block_table, "block_table", (B, max_pages), dev)
    lens = _ints(cache_lens, "cache_lens", (B,), dev)
    cu = None if cu_seqlens is None else _ints(cu_seqlens, "cu_seqlens", (B + 1,), dev)
    _run("s2attn_rope_append", dev, stream, lambda sm: lib().s2attn_rope_append(
        None if q is None else q.data_ptr(), None if q is None else q_rot.data_ptr(), k.data_ptr(),
        None if k_rot is None else k_rot.data_ptr(), v.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), table, cu, lens, T, B, Hq, Hkv, d, pages, page_size, max_pages, base,
        pi_scale, strides, sm))


def s2attn_decode_workspace_size(B, Hq, Hkv, d) -> int:
    return int(lib().s2attn_decode_workspace_size(B, Hq, Hkv, d))


def s2attn_decode(q, k_cache, v_cache, block_table, cache_lens, o, lse, scale=None, workspace=None,
                  stream=None):
    """Attention of one new token per sequence over the paged cache: q, o [B,Hq,d]; lse fp32 [B,Hq] or
    None; caches, block_table and cache_lens as in s2attn_rope_append. workspace: a uint8 CUDA tensor
    of s2attn_decode_workspace_size bytes that no other running call uses, or None to let torch
    allocate it."""
    dev = q.device
    B, Hq, d = q.shape
    pages, page_size, Hkv = k_cache.shape[:3]
    max_pages = block_table.shape[1]
    cache = (pages, page_size, Hkv, d)
    strides = (ctypes.c_longlong * 6)(
        _rows(q, "q", (B, Hq, d), dev), _rows(o, "o", (B, Hq, d), dev),
        *_cache_strides(k_cache, "k_cache", cache, dev), *_cache_strides(v_cache, "v_cache", cache, dev))
    table = _ints(block_table, "block_table", (B, max_pages), dev)
    lens = _ints(cache_lens, "cache_lens", (B,), dev)
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (B, Hq) or lse.device != dev
                            or not lse.is_contiguous()):
        raise ValueError(f"lse: expected a contiguous fp32 tensor of shape {(B, Hq)} on {dev}")
    if workspace is None:
        n = s2attn_decode_workspace_size(B, Hq, Hkv, d)
        with _on(stream, dev):
            workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous uint8 tensor on {dev}")
    _run("s2attn_decode", dev, stream, lambda sm: lib().s2attn_decode(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), table, lens, o.data_ptr(),
        None if lse is None else lse.data_ptr(), B, Hq, Hkv, d, pages, page_size, max_pages,
        d ** -0.5 if scale is None else scale, strides, workspace.data_ptr(), workspace.numel(), sm))


# ------------------------------------------------------------------------------------------
# Allocating conveniences
# ------------------------------------------------------------------------------------------
def rope_append(q, k, v, k_cache, v_cache, block_table, cache_lens, cu_seqlens=None, base=10000.0,
                pi_scale=1.0, stream=None):
    """s2attn_rope_append into new tensors: returns (q_rot, k_rot). Rows that are skipped (idle, or
    behind the last sequence) are left unset."""
    with _on(stream, k.device):
        q_rot, k_rot = torch.empty_like(q), torch.empty_like(k)
    s2attn_rope_append(q, q_rot, k, k_rot, v, k_cache, v_cache, block_table, cache_lens, cu_seqlens,
                       base, pi_scale, stream)
    return q_rot, k_rot


def decode(q, k_cache, v_cache, block_table, cache_lens, scale=None, stream=None):
    """s2attn_decode into new tensors: returns (o, lse)."""
    with _on(stream, q.device):
        o = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    s2attn_decode(q, k_cache, v_cache, block_table, cache_lens, o, lse, scale, None, stream)
    return o, lse
