"""CPU-side checks of the serving entries: argument validation in the library rejects bad calls before
any CUDA call (fake device addresses), and the Python binding refuses tensors it cannot pass on."""
import pytest
import torch

import shifted_sparse_attention_fwd_b200 as s2
from shifted_sparse_attention_fwd_b200 import build as s2build

A = 0x10000   # fake, 256-byte aligned device address: never dereferenced
OK, INVALID, UNSUPPORTED = 0, s2.S2ATTN_ERR_INVALID_ARG, s2.S2ATTN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    s2build.build()
    return s2.lib()


def _strides(*v):
    import ctypes
    return (ctypes.c_longlong * len(v))(*v)


def append_call(lib, **kw):
    a = dict(q=A, q_rot=A, k=A, k_rot=A, v=A, kc=A, vc=A, table=A, cu=A, lens=A, T=9, B=3, Hq=4, Hkv=2, d=64,
             pages=5, page_size=16, max_pages=2, base=1e4, pi=1.0, strides=None)
    a.update(kw)
    return lib.s2attn_rope_append(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(q_rot=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(k=A + 8), INVALID), (dict(k_rot=A + 2), INVALID), (dict(kc=A + 4), INVALID),
    (dict(T=0), INVALID), (dict(B=0), INVALID), (dict(cu=None), INVALID),   # T != B without cu_seqlens
    (dict(Hq=3), INVALID), (dict(Hkv=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
    (dict(pages=0), INVALID), (dict(page_size=0), INVALID), (dict(max_pages=-1), INVALID),
    (dict(page_size=1 << 20, max_pages=1 << 11), UNSUPPORTED),
    (dict(base=1.0), INVALID), (dict(base=float("inf")), INVALID), (dict(pi=0.0), INVALID),
    (dict(pi=float("nan")), INVALID),
    (dict(strides=_strides(252, 256, 128, 128, 128, 2048, 128, 2048, 128)), INVALID),   # not of 8
    (dict(strides=_strides(256, 248, 128, 128, 128, 2048, 128, 2048, 128)), INVALID),   # rows overlap
    (dict(strides=_strides(256, 256, 128, 128, 120, 2048, 128, 2048, 128)), INVALID),
    (dict(strides=_strides(256, 256, 128, 128, 128, 2040, 128, 2048, 128)), INVALID),   # pages overlap
    (dict(strides=_strides(256, 256, 128, 128, 128, 2048, 128, 2048, 64)), INVALID),
    (dict(strides=_strides(256, 256, 128, 128, 128, 2048, 128, -2048, 128)), INVALID),
])
def test_append_rejects(lib, kw, status):
    assert append_call(lib, **kw) == status


def decode_call(lib, **kw):
    a = dict(q=A, kc=A, vc=A, table=A, lens=A, o=A, lse=A, B=3, Hq=4, Hkv=2, d=64, pages=5, page_size=16,
             max_pages=2, scale=0.125, strides=None, ws=A, ws_bytes=1 << 30)
    a.update(kw)
    return lib.s2attn_decode(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(table=None), INVALID),
    (dict(lens=None), INVALID), (dict(o=None), INVALID), (dict(ws=None), INVALID), (dict(ws=A + 128), INVALID),
    (dict(ws_bytes=1024), INVALID), (dict(o=A + 8), INVALID), (dict(vc=A + 2), INVALID), (dict(B=0), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(Hq=5), INVALID), (dict(d=32), UNSUPPORTED), (dict(pages=0), INVALID), (dict(page_size=-4), INVALID),
    (dict(page_size=1 << 16, max_pages=1 << 15), UNSUPPORTED), (dict(B=1 << 30, Hq=4), UNSUPPORTED),
    (dict(strides=_strides(256, 256, 2048, 128, 2048, 100)), INVALID),
    (dict(strides=_strides(128, 256, 2048, 128, 2048, 128)), INVALID),
    (dict(strides=_strides(256, 260, 2048, 128, 2048, 128)), INVALID),
])
def test_decode_rejects(lib, kw, status):
    assert decode_call(lib, **kw) == status


def test_decode_workspace(lib):
    f = lib.s2attn_decode_workspace_size
    assert f(0, 4, 2, 64) == 0 and f(1, 4, 3, 64) == 0 and f(1, 4, 2, 96) == 0 and f(1, 0, 1, 64) == 0
    # proportional to the query heads of a kv head, up to one MMA's 16 rows; not to the batch
    assert 0 < f(1, 8, 8, 128) < f(1, 16, 8, 128) < f(1, 128, 8, 128) == f(9, 1024, 8, 128)
    assert f(1, 128, 8, 128) < 13 << 20


def prompt_call(lib, cu=(0, 100, 100, 256), **kw):
    import ctypes
    a = dict(q=A, k=A, v=A, o=A, lse=A, cu=(ctypes.c_int * len(cu))(*cu) if cu else None, n=len(cu or ()) - 1,
             T=256, Hq=4, Hkv=2, d=64, scale=0.125, strides=None)
    a.update(kw)
    return lib.s2attn_prompt_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID),
    (dict(lse=None), INVALID), (dict(cu=None), INVALID), (dict(q=A + 8), INVALID), (dict(o=A + 2), INVALID),
    (dict(n=0), INVALID), (dict(T=0), INVALID), (dict(T=255), INVALID), (dict(cu=(-1, 5)), INVALID),
    (dict(cu=(0, 9, 8, 20)), INVALID), (dict(cu=(0, 300, 200)), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(Hkv=3), INVALID), (dict(d=80), UNSUPPORTED),
    (dict(T=(1 << 23) + 1), UNSUPPORTED), (dict(Hq=1 << 20, Hkv=1), UNSUPPORTED),
    (dict(strides=_strides(256, 128, 128, 250)), INVALID), (dict(strides=_strides(256, 120, 128, 256)), INVALID),
])
def test_prompt_rejects(lib, kw, status):
    assert prompt_call(lib, **kw) == status


def test_binding_refuses_cpu_tensors_types_and_shapes():
    """The binding checks before it passes addresses on."""
    def t(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype)
    q, k, kc = t(3, 4, 64), t(3, 2, 64), t(5, 16, 2, 64)
    table, lens = t(3, 2, dtype=torch.int32), t(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        s2.rope_append(q, k, k.clone(), kc, kc.clone(), table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        s2.decode(q, kc, kc.clone(), table, lens)
    with pytest.raises(ValueError, match="float32"):
        s2.decode(q.float(), kc, kc.clone(), table, lens)
    with pytest.raises(ValueError, match="go together"):
        s2.s2attn_rope_append(q, None, k, None, k, kc, kc, table, lens)


def test_binding_is_loud_when_missing_or_of_another_torch(lib, monkeypatch, tmp_path):
    from shifted_sparse_attention_fwd_b200 import _serve
    monkeypatch.setattr(_serve, "BINDING_PATH", str(tmp_path / "none.so"))
    with pytest.raises(RuntimeError, match="build it"):
        _serve._load()
    monkeypatch.undo()
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    with pytest.raises(RuntimeError, match="build it again"):
        _serve._load()
