"""The serving entries of libs2attn.so for torch tensors: rotation and append to a paged key/value cache,
decode over it, and attention over packed prompts (include/s2attn.h, "Serving").

The checks of a call's tensors, its allocations and the call itself are in _s2torch.so
(csrc/s2_torch.cpp), a few microseconds less than they take here; there is no other path. Wrong tensors
raise ValueError, a failed call S2AttnError. Tensors on another device than the current one run there, on
that device's current stream; `stream` (a torch.cuda.Stream or a handle) overrides it. Views with
contiguous (heads, d) blocks are accepted wherever a tensor of heads is. A call of no rows (a scheduler's
empty step: no new tokens, no sequences to decode) launches nothing and returns empty tensors. There is no
backward: tensors that require grad are refused unless under torch.no_grad or inference_mode.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

from ._lib import S2AttnError, _stream, lib

BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_s2torch.so")

_binding = None


def _load():
    """_s2torch.so, bound to the loaded library; raises if it is missing or of another torch."""
    global _binding
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"{BINDING_PATH} is missing: build it with "
                           "`python -m shifted_sparse_attention_fwd_b200.build`")
    from . import _s2torch
    if _s2torch.TORCH_VERSION != torch.__version__.split("+")[0]:
        raise RuntimeError(f"{BINDING_PATH} was built for torch {_s2torch.TORCH_VERSION}, this is "
                           f"{torch.__version__}: build it again")
    handle = lib()
    _s2torch.bind(*(ctypes.cast(getattr(handle, name), ctypes.c_void_p).value for name in (
        "s2attn_rope_append_f64", "s2attn_decode", "s2attn_decode_workspace_size", "s2attn_prompt_fwd")))
    _binding = _s2torch
    return _s2torch


def _raise(status, name):
    raise S2AttnError(status, name)


def s2attn_rope_append(q, q_rot, k, k_rot, v, k_cache, v_cache, block_table, cache_lens,
                       cu_seqlens=None, base=10000.0, pi_scale=1.0, stream=None):
    """Turn the new tokens' q [T,Hq,d] into q_rot (both may be None; q_rot may be q) and k [T,Hkv,d]
    into the paged cache (and k_rot unless None; may be k), and copy v [T,Hkv,d] into the cache.
    k_cache, v_cache [pages,page_size,Hkv,d]; block_table int32 [B,max_pages]; cache_lens int32 [B],
    the tokens of each sequence including the new ones; cu_seqlens int32 [B+1], the sequences' first
    rows, or None for one new token per sequence. base and pi_scale are taken as Python floats, in 64 bits
    (the library's s2attn_rope_append_f64). A bad page or length on the device is reported by
    s2attn_get_device_error."""
    status = (_binding or _load()).rope_append(
        False, q, q_rot, k, k_rot, v, k_cache, v_cache, block_table, cache_lens, cu_seqlens, base, pi_scale,
        None if stream is None else _stream(stream))
    if status is not None:
        _raise(status, "s2attn_rope_append")


@functools.lru_cache(maxsize=256)
def s2attn_decode_workspace_size(B, Hq, Hkv, d) -> int:
    return int(lib().s2attn_decode_workspace_size(B, Hq, Hkv, d))


def s2attn_decode(q, k_cache, v_cache, block_table, cache_lens, o, lse, scale=None, workspace=None,
                  stream=None):
    """Attention of one new token per sequence over the paged cache: q, o [B,Hq,d]; lse fp32 [B,Hq] or
    None; caches, block_table and cache_lens as in s2attn_rope_append. workspace: a uint8 CUDA tensor
    of s2attn_decode_workspace_size bytes that no other running call uses, or None to let torch
    allocate it."""
    status = (_binding or _load()).decode(
        False, q, k_cache, v_cache, block_table, cache_lens, o, lse, scale, workspace,
        None if stream is None else _stream(stream))
    if status is not None:
        _raise(status, "s2attn_decode")


def _host_ints(cu_seqlens):
    if isinstance(cu_seqlens, torch.Tensor):
        return cu_seqlens
    return torch.tensor(cu_seqlens, dtype=torch.int32, device="cpu")   # (whatever torch's default device is)


def s2attn_prompt_fwd(q, k, v, o, lse, cu_seqlens, scale=None, stream=None):
    """Causal attention over packed prompts: q, o [T,Hq,d], k, v [T,Hkv,d] bf16; lse fp32 [Hq,T].
    cu_seqlens: the sequences' first rows and the end of the last, on the HOST (a contiguous int32 CPU
    tensor, or a sequence of ints)."""
    status = (_binding or _load()).prompt_fwd(
        False, q, k, v, o, lse, _host_ints(cu_seqlens), scale, None if stream is None else _stream(stream))
    if status is not None:
        _raise(status, "s2attn_prompt_fwd")


# ------------------------------------------------------------------------------------------
# Allocating conveniences
# ------------------------------------------------------------------------------------------
def rope_append(q, k, v, k_cache, v_cache, block_table, cache_lens, cu_seqlens=None, base=10000.0,
                pi_scale=1.0, stream=None):
    """s2attn_rope_append into new tensors: returns (q_rot, k_rot). Rows that are skipped (idle, or
    behind the last sequence) are left unset."""
    out = (_binding or _load()).rope_append(
        True, q, None, k, None, v, k_cache, v_cache, block_table, cache_lens, cu_seqlens, base, pi_scale,
        None if stream is None else _stream(stream))
    return out if type(out) is tuple else _raise(out, "s2attn_rope_append")


def decode(q, k_cache, v_cache, block_table, cache_lens, scale=None, stream=None):
    """s2attn_decode into new tensors: returns (o, lse)."""
    out = (_binding or _load()).decode(
        True, q, k_cache, v_cache, block_table, cache_lens, None, None, scale, None,
        None if stream is None else _stream(stream))
    return out if type(out) is tuple else _raise(out, "s2attn_decode")


def prompt_fwd(q, k, v, cu_seqlens, scale=None, stream=None):
    """s2attn_prompt_fwd into new tensors: returns (o, lse). Rows of no sequence are left unset."""
    out = (_binding or _load()).prompt_fwd(
        True, q, k, v, None, None, _host_ints(cu_seqlens), scale, None if stream is None else _stream(stream))
    return out if type(out) is tuple else _raise(out, "s2attn_prompt_fwd")
