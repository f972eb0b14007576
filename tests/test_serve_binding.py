"""CPU-side checks of the serving entries' Python face and of what the library answers without a GPU."""
import pytest
import torch

import shifted_sparse_attention_fwd_b200 as s2
from shifted_sparse_attention_fwd_b200 import build as s2build


@pytest.fixture(scope="module")
def lib():
    s2build.build()
    return s2.lib()


def test_decode_workspace_is_0_for_every_call_that_decode_rejects(lib):
    """Also for batches of 2^31 rows and more, which s2attn_decode has no room to number."""
    f = lib.s2attn_decode_workspace_size
    assert f(1 << 29, 4, 2, 64) == 0 and f((1 << 31) - 1, 2, 2, 128) == 0
    assert f((1 << 29) - 1, 4, 2, 64) == f(1, 4, 2, 64) > 0


def _append_f64(lib, base, pi):
    A = 0x10000   # fake device address: never dereferenced
    return lib.s2attn_rope_append_f64(*[A] * 10, 9, 3, 4, 2, 64, 5, 16, 2, base, pi, None, None)


@pytest.mark.parametrize("base,pi", [(1.0, 0.5), (float("inf"), 0.5), (float("nan"), 0.5), (1e4, 0.0), (1e4, -0.3),
                                     (1e4, float("nan")), (1e4, float("inf"))])
def test_append_f64_rejects(lib, base, pi):
    assert _append_f64(lib, base, pi) == s2.S2ATTN_ERR_INVALID_ARG


def test_lengths_given_as_ints_stay_on_the_host():
    """prompt_fwd takes a list of ints under any default device of torch's."""
    from shifted_sparse_attention_fwd_b200 import _serve
    with torch.device("meta"):
        cu = _serve._host_ints([0, 5, 9])
    assert cu.device.type == "cpu" and cu.dtype == torch.int32 and cu.tolist() == [0, 5, 9]


def test_build_makes_the_binding_again_for_another_torch(lib, monkeypatch, tmp_path):
    """The binding fits one torch only and refuses to load with another, so build() follows the torch that is
    installed, not the files' times alone."""
    import os
    compiled = []

    def compile_(cmd, out, verbose):
        compiled.append(out)
        with open(out, "w"):
            pass
    monkeypatch.setattr(s2build, "_compile", compile_)
    monkeypatch.setattr(s2build, "BINDING", str(tmp_path / "b.so"))
    monkeypatch.setattr(s2build, "BINDING_TORCH", str(tmp_path / "x" / "version"), raising=False)
    s2build.build_binding()
    s2build.build_binding()
    assert compiled == [str(tmp_path / "b.so")]
    monkeypatch.setattr(torch, "__version__", "1.0.0+cu1")
    s2build.build_binding()
    s2build.build_binding()
    assert len(compiled) == 2
    os.remove(tmp_path / "b.so")
    s2build.build_binding()
    assert len(compiled) == 3
