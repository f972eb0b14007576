"""Binding of the serving entries of libs2attn.so: rotation and append to a paged key/value cache,
decode over it, and attention over packed prompts (include/s2attn.h, "Serving").

Argument marshalling only, as in _lib.py. A decoding step is a few microseconds of GPU work, so
these functions keep their own cost low: one pass over the arguments and one ctypes call. Tensors
that belong to another device than the current one are run on that device's current stream.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._lib import S2ATTN_OK, S2AttnError, _stream, lib

_BF16, _I32 = torch.bfloat16, torch.int32
_raw_stream = torch._C._cuda_getCurrentRawStream   # the current stream's handle, by device index
_get_device = torch._C._cuda_getDevice


def _owner(stream, device):
    """Context in which the tensors of a call are allocated: they belong to the stream it runs on."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _like(t, stream):
    """A new contiguous tensor of t's shape and type."""
    if stream is None:
        return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)
    with _owner(stream, t.device):
        return t.new_empty(t.shape)


def _new(t, shape, dtype, stream):
    if stream is None:
        return t.new_empty(shape, dtype=dtype)
    with _owner(stream, t.device):
        return t.new_empty(shape, dtype=dtype)


def _run(name, index, stream, args):
    """The C function on device `index`, which is made current, with the stream's handle last."""
    fn = getattr(lib(), name)
    if index == _get_device():
        status = fn(*args, _raw_stream(index) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index) if stream is None else _stream(stream))
    if status != S2ATTN_OK:
        raise S2AttnError(status, name)


def _check(name, t, dtype, shape, index):
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if index < 0 or t.get_device() != index:
        raise ValueError(f"{name}: expected a CUDA tensor on device {index}, got {t.device}")


def _tensors(index, *named):
    """Checks the (name, bf16 tensor or None, shape) of a call; whether all are contiguous."""
    packed = True
    for name, t, shape in named:
        if t is None:
            continue
        # one cheap test for the usual case; _check says what is wrong
        if t.dtype is not _BF16 or t.shape != shape or t.get_device() != index or index < 0:
            _check(name, t, _BF16, shape, index)
        packed = packed and t.is_contiguous()
    return packed


def _ints(index, name, t, shape):
    if t.dtype is not _I32 or t.shape != shape or t.get_device() != index:
        _check(name, t, _I32, shape, index)
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _outer_strides(name, t):
    """Strides of the axes before a tensor's contiguous (heads, d) block."""
    st = t.stride()
    if st[-1] != 1 or st[-2] != t.shape[-1]:
        raise ValueError(f"{name}: expected contiguous (heads, d) blocks")
    return st[:-2]


def s2attn_rope_append(q, q_rot, k, k_rot, v, k_cache, v_cache, block_table, cache_lens,
                       cu_seqlens=None, base=10000.0, pi_scale=1.0, stream=None):
    """Turn the new tokens' q [T,Hq,d] into q_rot (both may be None; q_rot may be q) and k [T,Hkv,d]
    into the paged cache (and k_rot unless None; may be k), and copy v [T,Hkv,d] into the cache.
    k_cache, v_cache [pages,page_size,Hkv,d]; block_table int32 [B,max_pages]; cache_lens int32 [B],
    the tokens of each sequence including the new ones; cu_seqlens int32 [B+1], the sequences' first
    rows, or None for one new token per sequence. Views with contiguous (heads, d) blocks are
    accepted. A bad page or length on the device is reported by s2attn_get_device_error."""
    index = k.get_device()
    T, Hkv, d = rows = k.shape
    pages, page_size = k_cache.shape[:2]
    B, max_pages = block_table.shape
    if (q is None) != (q_rot is None):
        raise ValueError("q and q_rot go together")
    Hq = Hkv if q is None else q.shape[1]
    q_shape, cache = (T, Hq, d), (pages, page_size, Hkv, d)
    named = (("q", q, q_shape), ("q_rot", q_rot, q_shape), ("k", k, rows), ("k_rot", k_rot, rows),
             ("v", v, rows), ("k_cache", k_cache, cache), ("v_cache", v_cache, cache))
    strides = None
    if not _tensors(index, *named):
        flat = []
        for (name, t, _), like in zip(named, (None, q, None, k, None, None, None)):
            flat += _outer_strides(name, t if t is not None else like if like is not None else k)
        strides = (ctypes.c_longlong * 9)(*flat)
    _run("s2attn_rope_append", index, stream, (
        None if q is None else q.data_ptr(), None if q is None else q_rot.data_ptr(), k.data_ptr(),
        None if k_rot is None else k_rot.data_ptr(), v.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), _ints(index, "block_table", block_table, (B, max_pages)),
        None if cu_seqlens is None else _ints(index, "cu_seqlens", cu_seqlens, (B + 1,)),
        _ints(index, "cache_lens", cache_lens, (B,)), T, B, Hq, Hkv, d, pages, page_size, max_pages,
        base, pi_scale, strides))


@functools.lru_cache(maxsize=256)
def s2attn_decode_workspace_size(B, Hq, Hkv, d) -> int:
    return int(lib().s2attn_decode_workspace_size(B, Hq, Hkv, d))


def s2attn_decode(q, k_cache, v_cache, block_table, cache_lens, o, lse, scale=None, workspace=None,
                  stream=None):
    """Attention of one new token per sequence over the paged cache: q, o [B,Hq,d]; lse fp32 [B,Hq] or
    None; caches, block_table and cache_lens as in s2attn_rope_append. workspace: a uint8 CUDA tensor
    of s2attn_decode_workspace_size bytes that no other running call uses, or None to let torch
    allocate it."""
    index = q.get_device()
    B, Hq, d = rows = q.shape
    pages, page_size, Hkv = k_cache.shape[:3]
    max_pages = block_table.shape[1]
    cache = (pages, page_size, Hkv, d)
    named = (("q", q, rows), ("o", o, rows), ("k_cache", k_cache, cache), ("v_cache", v_cache, cache))
    strides = None
    if not _tensors(index, *named):
        flat = []
        for name, t, _ in named:
            flat += _outer_strides(name, t)
        strides = (ctypes.c_longlong * 6)(*flat)
    if lse is not None:
        _check("lse", lse, torch.float32, (B, Hq), index)
        if not lse.is_contiguous():
            raise ValueError("lse: expected a contiguous tensor")
    if workspace is None:
        workspace = _new(q, s2attn_decode_workspace_size(B, Hq, Hkv, d), torch.uint8, stream)
    else:
        _check("workspace", workspace, torch.uint8, workspace.shape, index)
        if not workspace.is_contiguous():
            raise ValueError("workspace: expected a contiguous tensor")
    _run("s2attn_decode", index, stream, (
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        _ints(index, "block_table", block_table, (B, max_pages)),
        _ints(index, "cache_lens", cache_lens, (B,)), o.data_ptr(),
        None if lse is None else lse.data_ptr(), B, Hq, Hkv, d, pages, page_size, max_pages,
        d ** -0.5 if scale is None else scale, strides, workspace.data_ptr(), workspace.numel()))


def s2attn_prompt_fwd(q, k, v, o, lse, cu_seqlens, scale=None, stream=None):
    """Causal attention over packed prompts: q, o [T,Hq,d], k, v [T,Hkv,d] bf16; lse fp32 [Hq,T].
    cu_seqlens: the sequences' first rows and the end of the last, on the HOST (a contiguous int32 CPU tensor,
    or a sequence of ints). Views with contiguous (heads, d) blocks are accepted."""
    index = q.get_device()
    T, Hq, d = rows = q.shape
    Hkv = k.shape[1]
    kv = (T, Hkv, d)
    named = (("q", q, rows), ("k", k, kv), ("v", v, kv), ("o", o, rows))
    strides = None
    if not _tensors(index, *named):
        strides = (ctypes.c_longlong * 4)(*(x for name, t, _ in named for x in _outer_strides(name, t)))
    _check("lse", lse, torch.float32, (Hq, T), index)
    if not lse.is_contiguous():
        raise ValueError("lse: expected a contiguous tensor")
    if not isinstance(cu_seqlens, torch.Tensor):
        cu_seqlens = torch.tensor(cu_seqlens, dtype=_I32)
    if (cu_seqlens.is_cuda or cu_seqlens.dtype is not _I32 or cu_seqlens.dim() != 1
            or not cu_seqlens.is_contiguous()):
        raise ValueError("cu_seqlens: expected a contiguous int32 CPU tensor of one axis, or a sequence of ints")
    _run("s2attn_prompt_fwd", index, stream, (
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), cu_seqlens.data_ptr(),
        cu_seqlens.numel() - 1, T, Hq, Hkv, d, d ** -0.5 if scale is None else scale, strides))


# ------------------------------------------------------------------------------------------
# Allocating conveniences
# ------------------------------------------------------------------------------------------
def rope_append(q, k, v, k_cache, v_cache, block_table, cache_lens, cu_seqlens=None, base=10000.0,
                pi_scale=1.0, stream=None):
    """s2attn_rope_append into new tensors: returns (q_rot, k_rot). Rows that are skipped (idle, or
    behind the last sequence) are left unset."""
    q_rot, k_rot = _like(q, stream), _like(k, stream)
    s2attn_rope_append(q, q_rot, k, k_rot, v, k_cache, v_cache, block_table, cache_lens, cu_seqlens,
                       base, pi_scale, stream)
    return q_rot, k_rot


def decode(q, k_cache, v_cache, block_table, cache_lens, scale=None, stream=None):
    """s2attn_decode into new tensors: returns (o, lse)."""
    o, lse = _like(q, stream), _new(q, q.shape[:2], torch.float32, stream)
    s2attn_decode(q, k_cache, v_cache, block_table, cache_lens, o, lse, scale, None, stream)
    return o, lse


def prompt_fwd(q, k, v, cu_seqlens, scale=None, stream=None):
    """s2attn_prompt_fwd into new tensors: returns (o, lse). Rows of no sequence are left unset."""
    o, lse = _like(q, stream), _new(q, (q.shape[1], q.shape[0]), torch.float32, stream)
    s2attn_prompt_fwd(q, k, v, o, lse, cu_seqlens, scale, stream)
    return o, lse
