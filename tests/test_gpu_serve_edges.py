"""The serving operators on the GPU where a call is unusual. Tolerances as derived in test_gpu_serve.py, whose
helpers are used."""
import ctypes
import random

import pytest
import torch

import shifted_sparse_attention_fwd_b200 as s2
from test_gpu_serve import (BF16_STEP, _caches, _check_decode, _cu, _decode64, _ints, _near_bf16, _ok, _prompt64,
                            _randn, _table, _turn64)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    s2.lib()


# ------------------------------------------------------------------------------------------
# infinities and NaN in values that a row sees
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (8, 1, 64), (16, 2, 128), (9, 1, 64), (16, 1, 128), (17, 1, 64)])
@pytest.mark.parametrize("lens", [[1, 40, 300], [9000, 0, 77], [700] * 5])
def test_decode_infinite_and_nan_values(hq, hkv, d, lens):
    """A seen value of +inf makes its column +inf for every group size, opposite infinities and NaN make it NaN,
    and no other column moves. (Scores are small, so no weight underflows.)"""
    page = 16
    rows, pages = _table(lens, page, 7)
    kc, vc = _randn(1, pages, page, hkv, d), _randn(2, pages, page, hkv, d)
    q = _randn(3, len(lens), hq, d)
    table, n = _ints(rows), _ints(lens)
    want, want_lse = s2.decode(q, kc, vc, table, n)
    seen = torch.zeros(len(lens), hkv, d, dtype=torch.float64, device="cuda")
    for b, m in enumerate(lens):
        # (token, column, value): first and last token, the middle one, two of opposite signs
        for t, c, x in ((0, 0, "inf"), (m - 1, 1, "inf"), (m // 2, 2, "-inf"), (m // 3, d - 1, "nan"), (0, 5, "inf"),
                        (m - 1, 5, "-inf" if m > 1 else "inf"), (m // 2, 8, "inf"), (m // 4, 8, "inf")):
            if m:
                h = (b + c) % hkv
                if vc[rows[b][t // page], t % page, h, c].isfinite():
                    vc[rows[b][t // page], t % page, h, c] = float(x)
                    seen[b, h, c] += float(x)
    o, lse = s2.decode(q, kc, vc, table, n)
    _ok()
    assert torch.equal(lse, want_lse)
    seen = seen.repeat_interleave(hq // hkv, 1)
    clean = seen == 0
    assert torch.equal(o[clean], want[clean])
    got = o.double()
    assert torch.equal(got[seen.isinf()], seen[seen.isinf()]) and got[seen.isnan()].isnan().all()


def _us(call):
    """Device time of one call, the best of five."""
    best = float("inf")
    call()
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (3, 3, 64)])
@pytest.mark.parametrize("x", ["nan", "inf", "-inf"])
def test_prompt_of_nothing_but_infinite_values(hq, hkv, d, x):
    """An overflowed layer's values: every result is what the formula gives, in a time of the same order as
    with finite values (walking them value by value took hundreds of times as long)."""
    cu = torch.tensor([0, 1200, 1201, 1300], dtype=torch.int32)
    q, k, v = (_randn(60 + i, 1300, h, d) for i, h in enumerate((hq, hkv, hkv)))
    o, lse = torch.empty_like(q), torch.empty(hq, 1300, device="cuda")
    s2.s2attn_prompt_fwd(q, k, v, o, lse, cu)
    want_lse = lse.clone()
    plain = _us(lambda: s2.s2attn_prompt_fwd(q, k, v, o, lse, cu))
    v.fill_(float(x))
    full = _us(lambda: s2.s2attn_prompt_fwd(q, k, v, o, lse, cu))
    _ok()
    assert torch.equal(lse, want_lse)
    assert o.isnan().all() if x == "nan" else (o == float(x)).all()
    # a unit's 256 rows are read and written once more, by one warp: about 40 us beside its 10 to 20
    assert full <= 16 * plain + 50, (plain, full)


# ------------------------------------------------------------------------------------------
# lengths and pages outside the cache
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("lens,cu,skipped", [
    ([3, -1], None, [1]),                        # one token each, a negative length
    ([3, -(1 << 31)], None, [1]),
    ([3, -5], [0, 2, 5], [2, 3, 4]),             # several rows of a sequence of a negative length
    ([3, 2], [0, 2, 5], [2]),                    # a length that leaves the new rows out: the first has no position
    ([3, 1], [0, 2, 5], [2, 3]),
])
def test_append_reports_lengths_too_small_for_the_rows(lens, cu, skipped):
    """Rows without a position are skipped, and reported unless the sequence is idle (length 0)."""
    page, hq, hkv, d = 8, 4, 2, 64
    T = cu[-1] if cu else 2
    q, k, v = (_randn(1 + i, T, h, d) for i, h in enumerate((hq, hkv, hkv)))
    kc, vc = _randn(4, 2, page, hkv, d), _randn(5, 2, page, hkv, d)
    kc0, vc0 = kc.clone(), vc.clone()
    q_rot, k_rot = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    table = _ints([[0], [1]])
    args = (q, q_rot, k, k_rot, v, kc, vc, table)
    cu_dev = None if cu is None else _ints(cu)
    s2.s2attn_rope_append(*args, _ints(lens), cu_dev)
    torch.cuda.synchronize()
    assert s2.s2attn_get_device_error() == (s2.S2ATTN_ERR_INVALID_ARG, (6 << 8) | 0x81)
    rows = [(s, t) for s in range(2) for t in (range(cu[s], cu[s + 1]) if cu else [s])]
    for s, t in rows:
        if t in skipped:
            assert (q_rot[t] == 7).all() and (k_rot[t] == 7).all()
            continue
        pos = lens[s] - (cu[s + 1] if cu else s + 1) + t
        kc0[s, pos], vc0[s, pos] = k_rot[t], v[t]
        _near_bf16(k_rot[t:t + 1], _turn64(k[t:t + 1], torch.tensor([pos], device="cuda"), 10000.0, 1.0), 1.2e-5)
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)
    # an idle sequence is no error
    s2.s2attn_rope_append(*args, _ints([3, 0]), cu_dev)
    _ok()


@pytest.mark.parametrize("width", [2, 70])       # whole segments; the list form, which splits (70 x 16 tokens)
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (16, 1, 128)])
def test_decode_bad_pages_count_as_zeros_and_lengths_are_cut(width, hq, hkv, d):
    page, B = 16, 3
    n = width * page - 3
    pages = 3 * width
    kc, vc = _randn(2, pages, page, hkv, d), _randn(3, pages, page, hkv, d)
    q = _randn(1, B, hq, d)
    good = [list(range(b * width, (b + 1) * width)) for b in range(B)]

    def reference(table, lens):
        """Tokens of a bad page: keys and values of zeros, in two more pages behind the cache's own."""
        k0, v0 = (torch.cat((x, torch.zeros(1, page, hkv, d, dtype=x.dtype, device="cuda"))) for x in (kc, vc))
        rows = [[x if 0 <= x < pages else pages for x in r] for r in table]
        return k0, v0, rows, [min(max(m, 0), width * page) for m in lens]

    for bad, lens, site in ((pages, [n, n, n], 0x80), (-1, [n, n, n], 0x80), (1 << 30, [n, 5, n], 0x80),
                            (None, [n, width * page + 1, 7], 0x81), (None, [n, -1, (1 << 31) - 1], 0x81)):
        table = [list(r) for r in good]
        if bad is not None:
            table[1][0] = table[2][width - 1] = bad
        o, lse = s2.decode(q, kc, vc, _ints(table), _ints(lens))
        torch.cuda.synchronize()
        assert s2.s2attn_get_device_error() == (s2.S2ATTN_ERR_INVALID_ARG, (7 << 8) | site)
        k0, v0, rows, cut = reference(table, lens)
        _check_decode(q, k0, v0, rows, cut, d ** -0.5, o, lse)


# ------------------------------------------------------------------------------------------
# scales that fp32 does not hold
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("base,pi", [(10000.0, 0.3), (10000.0, 4096 / 100000), (500000.7, 1 / 3), (1e6, 0.1)])
def test_append_angles_of_any_scale_at_far_positions(base, pi):
    """base and pi_scale are Python floats; the angle is that of their product, not of its fp32 neighbour
    (0.3 in fp32 is off by 1.6e-3 rad at position 131071)."""
    hq, hkv, d, page = 2, 1, 128, 1 << 12
    pos = [131071, 131072 - 4096, 99999, 65537, 1, 0]
    k, q, v = (_randn(7 + i, len(pos), h, d) for i, h in enumerate((hkv, hq, hkv)))
    kc, vc = _randn(1, len(pos), page, hkv, d), _randn(2, len(pos), page, hkv, d)
    table = _ints([[b] * 32 for b in range(len(pos))])
    q_rot, k_rot = s2.rope_append(q, k, v, kc, vc, table, _ints([p + 1 for p in pos]), base=base, pi_scale=pi)
    _ok()
    at = torch.tensor(pos, device="cuda")
    _near_bf16(q_rot, _turn64(q, at, base, pi), 1.2e-5)
    _near_bf16(k_rot, _turn64(k, at, base, pi), 1.2e-5)


# ------------------------------------------------------------------------------------------
# empty calls
# ------------------------------------------------------------------------------------------
def test_empty_calls_return_empty_tensors():
    """A scheduler's empty step: no new rows, no sequences. Nothing is launched or written."""
    hq, hkv, d, page = 8, 2, 64, 16
    kc, vc = _randn(1, 3, page, hkv, d), _randn(2, 3, page, hkv, d)
    kc0, vc0 = kc.clone(), vc.clone()
    q, k = _randn(3, 0, hq, d), _randn(4, 0, hkv, d)
    none = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    some, lens = _ints([[0, 1], [2, 2]]), _ints([5, 0])
    for table, n, cu in ((none, _ints([]), None), (none, _ints([]), _ints([0])), (some, lens, _ints([0, 0, 0]))):
        q_rot, k_rot = s2.rope_append(q, k, k, kc, vc, table, n, cu)
        assert q_rot.shape == q.shape and k_rot.shape == k.shape and q_rot.dtype == torch.bfloat16
        q_rot, k_rot = s2.rope_append(None, k, k, kc, vc, table, n, cu)
        assert q_rot is None and k_rot.shape == k.shape
        s2.s2attn_rope_append(q, q, k, None, k, kc, vc, table, n, cu)
    o, lse = s2.decode(q, kc, vc, none, _ints([]))
    assert o.shape == (0, hq, d) and lse.shape == (0, hq) and lse.dtype == torch.float32
    s2.s2attn_decode(q, kc, vc, none, _ints([]), o, None)
    for cu in ([0], [0, 0], torch.zeros(4, dtype=torch.int32)):
        o, lse = s2.prompt_fwd(q, k, k, cu)
        assert o.shape == q.shape and lse.shape == (hq, 0)
        s2.s2attn_prompt_fwd(q, k, k, o, lse, cu)
    _ok()
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)
    # what is wrong in a call of some rows is wrong in one of none
    with pytest.raises(s2.S2AttnError, match="invalid"):
        s2.rope_append(q, k, k, kc, vc, some, lens)                       # T != B and no cu_seqlens
    with pytest.raises(s2.S2AttnError, match="invalid"):
        s2.prompt_fwd(q, k, k, [0, 1])
    with pytest.raises(s2.S2AttnError, match="invalid"):
        s2.prompt_fwd(q, k, k, [])
    with pytest.raises(s2.S2AttnError, match="invalid"):
        s2.decode(_randn(1, 0, 3, d), kc, vc, none, _ints([]))            # 3 query heads over 2
    with pytest.raises(s2.S2AttnError, match="unsupported"):
        s2.prompt_fwd(_randn(1, 0, 4, 96), _randn(1, 0, 2, 96), _randn(1, 0, 2, 96), [0])
    with pytest.raises(s2.S2AttnError, match="invalid"):
        s2.decode(q, kc, vc, none, _ints([]), scale=-1.0)
    with pytest.raises(s2.S2AttnError, match="invalid"):
        s2.rope_append(q, k, k, kc, vc, none, _ints([]), pi_scale=0.0)


# ------------------------------------------------------------------------------------------
# autograd
# ------------------------------------------------------------------------------------------
def _small():
    hq, hkv, d, page = 4, 2, 64, 8
    t = dict(q=_randn(1, 2, hq, d), k=_randn(2, 2, hkv, d), v=_randn(3, 2, hkv, d),
             k_cache=_randn(4, 3, page, hkv, d), v_cache=_randn(5, 3, page, hkv, d))
    return t, _ints([[0], [2]]), _ints([3, 8])


@pytest.mark.parametrize("name", ["q", "k", "v", "k_cache", "v_cache"])
def test_tensors_that_need_a_gradient_are_refused(name):
    """There is no backward: a graph that would end at the call is refused, not cut in silence. Under
    torch.no_grad the same tensors are fine, and give the same result."""
    t, table, lens = _small()
    plain = {n: x.clone() for n, x in t.items()}
    t[name].requires_grad_()

    def calls(t):
        yield "append", lambda: s2.rope_append(t["q"], t["k"], t["v"], t["k_cache"], t["v_cache"], table, lens)
        yield "decode", lambda: s2.decode(t["q"], t["k_cache"], t["v_cache"], table, lens)
        yield "prompt", lambda: s2.prompt_fwd(t["q"], t["k"], t["v"], [0, 2])
    uses = {"append": ("q", "k", "v", "k_cache", "v_cache"), "decode": ("q", "k_cache", "v_cache"),
            "prompt": ("q", "k", "v")}
    for (op, call), (_, want) in zip(calls(t), calls(plain)):
        if name in uses[op]:
            with pytest.raises(ValueError, match=f"{name}: requires grad"):
                call()
        with torch.no_grad():
            for x, y in zip(call(), want()):
                assert torch.equal(x, y) and not x.requires_grad
        with torch.inference_mode():
            call()
    _ok()
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(plain["q"], torch.ones_like(plain["q"]))
        with pytest.raises(ValueError, match="q: .*tangent"):
            s2.decode(dual, plain["k_cache"], plain["v_cache"], table, lens)


def test_writes_raise_the_version_of_what_they_write():
    """Autograd's check for tensors changed in place sees the caches and the outputs that a call is given; what
    it only reads keeps its version. Tensors of inference mode, which have none, can be written."""
    t, table, lens = _small()
    q, k, v, kc, vc = t.values()
    o, lse = torch.empty_like(q), torch.empty(2, 4, device="cuda")
    plse = torch.empty(4, 2, device="cuda")

    def versions():
        return [x._version for x in (q, k, v, kc, vc, o, lse, plse, table, lens)]
    a = versions()
    s2.rope_append(q, k, v, kc, vc, table, lens)
    b = versions()
    assert [y - x for x, y in zip(a, b)] == [0, 0, 0, 1, 1, 0, 0, 0, 0, 0]
    s2.s2attn_rope_append(q, q, k, k, v, kc, vc, table, lens)
    c = versions()
    assert [y - x for x, y in zip(b, c)] == [1, 1, 0, 1, 1, 0, 0, 0, 0, 0]
    s2.s2attn_decode(q, kc, vc, table, lens, o, lse)
    d = versions()
    assert [y - x for x, y in zip(c, d)] == [0, 0, 0, 0, 0, 1, 1, 0, 0, 0]
    s2.s2attn_prompt_fwd(q, k, v, o, plse, [0, 2])
    assert [y - x for x, y in zip(d, versions())] == [0, 0, 0, 0, 0, 1, 0, 1, 0, 0]
    half = torch.ones(1, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    y = (half * kc).sum()                              # a graph that holds the cache
    s2.rope_append(q, k, v, kc, vc, table, lens)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        ki, vi = kc.clone(), vc.clone()
    s2.rope_append(q, k, v, ki, vi, table, lens)
    _ok()


# ------------------------------------------------------------------------------------------
# a failed launch
# ------------------------------------------------------------------------------------------
def test_a_failed_launch_is_not_the_next_call_s_error():
    """A launch into a stream whose capture has been broken off fails on the host, before anything reaches the
    GPU. The call that failed says so; the calls after it are not told again."""
    rt = ctypes.CDLL("libcudart.so.12")                # the runtime that torch has loaded
    side = torch.cuda.Stream()
    handle = ctypes.c_void_p(side.cuda_stream)
    q = _randn(1, 64, 2, 64).unsqueeze(0)
    p = q[0]
    want = s2.fwd(q, q, q, 64)
    o, lse = torch.empty_like(p), torch.empty(2, 64, device="cuda")
    s2.s2attn_prompt_fwd(p, p, p, o, lse, [0, 64])
    torch.cuda.synchronize()
    graph = ctypes.c_void_p()
    assert rt.cudaStreamBeginCapture(handle, 1) == 0                      # thread-local mode
    try:
        assert rt.cudaStreamSynchronize(handle) != 0                      # breaks the capture off
        with pytest.raises(s2.S2AttnError, match="launch"):
            s2.s2attn_prompt_fwd(p, p, p, o, lse, [0, 64], stream=side)
    finally:
        rt.cudaStreamEndCapture(handle, ctypes.byref(graph))
        rt.cudaGetLastError()
    got = s2.fwd(q, q, q, 64)
    _ok()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------------------------------
# large values
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (3, 3, 64)])
def test_prompt_values_up_to_the_stated_limit(hq, hkv, d):
    """Values just below 2^98 / ceil(n / 128) under scores that grow to almost 2^30 in a tile's sum over a row's
    first 16 (so the passes are not repeated): finite, and right."""
    n = 500
    q, k, v = (_randn(80 + i, n, h, d) for i, h in enumerate((hq, hkv, hkv)))
    # the score of key r is 16 r / n nats: its weight over the first ones' 2^(23 r / n), a last tile's sum 2^28
    q.fill_(1.0)
    k.copy_((torch.arange(n, device="cuda") * (16.0 / n))[:, None, None].expand_as(k))
    v.copy_((v.float().abs().clamp(0.5, 1.98) * 2.0 ** 95).to(torch.bfloat16))
    cu = [0, n]
    o, lse = s2.prompt_fwd(q, k, v, cu, scale=1.0 / d)
    _ok()
    want, want_lse, mean_abs = _prompt64(q, k, v, cu, 1.0 / d)
    _near_bf16(o, want, (BF16_STEP + 1e-5) * mean_abs)
    assert float((lse.double() - want_lse).abs().max()) <= 2e-5


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (12, 1, 64)])
@pytest.mark.parametrize("n", [400, 1000])
def test_decode_values_up_to_the_stated_limit(hq, hkv, d, n):
    """Values just below 2^120 / n under scores that grow slowly, so that the sums keep a reference of up to 2^8
    below them."""
    page, lens = 16, [n, 1]
    rows, pages = _table(lens, page, 4)
    kc, vc = _randn(1, pages, page, hkv, d), _randn(2, pages, page, hkv, d)
    q = torch.ones(2, hq, d, dtype=torch.bfloat16, device="cuda")
    vc.copy_((vc.float().abs().clamp(0.5, 1.98) * 2.0 ** 109).to(torch.bfloat16))
    t = torch.arange(n, device="cuda")
    kc[torch.tensor(rows[0], device="cuda")[t // page], t % page] = (t * (16.0 / n))[:, None, None].to(torch.bfloat16)
    o, lse = s2.decode(q, kc, vc, _ints(rows), _ints(lens), scale=1.0 / d)
    _ok()
    _check_decode(q, kc, vc, rows, lens, 1.0 / d, o, lse)


# ------------------------------------------------------------------------------------------
# captured steps with other work between
# ------------------------------------------------------------------------------------------
def test_captured_steps_between_copies_fills_and_other_streams():
    """The kernels may start before the work in front of them has ended, and wait for it: copies, fills, torch's
    own kernels and a fork onto a second stream, captured and replayed, and queued without a capture."""
    hq, hkv, d, page, B, width = 8, 2, 128, 16, 4, 40
    kc, vc = _randn(1, B * width, page, hkv, d), _randn(2, B * width, page, hkv, d)
    rows = [list(range(b * width, (b + 1) * width)) for b in range(B)]
    table, lens = torch.zeros(B, width, dtype=torch.int32, device="cuda"), _ints([0] * B)
    src = {"table": _ints(rows), "lens": _ints([599, 17, 0, 320]), "q": _randn(3, B, hq, d), "k": _randn(4, B, hkv, d),
           "v": _randn(5, B, hkv, d)}
    q, k, v = (torch.empty_like(src[x]) for x in "qkv")
    cu = [0, 1, 4]
    step = torch.ones(B, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    out = {}

    def steps():
        table.zero_()                                  # a fill
        table.copy_(src["table"])                      # copies
        lens.copy_(src["lens"])
        for x, y in ((q, "q"), (k, "k"), (v, "v")):
            x.copy_(src[y])
        lens.add_(step)                                # a kernel
        q_rot, k_rot = s2.rope_append(q, k, v, kc, vc, table, lens)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            po, plse = s2.prompt_fwd(q_rot, k_rot, v, cu)
            scaled = po.float() * 2                    # torch's own kernel behind ours
        o, lse = s2.decode(q_rot, kc, vc, table, lens)
        total = o.float().sum(-1)
        torch.cuda.current_stream().wait_stream(side)
        lens.zero_()                                   # behind the last kernel that reads it
        q.fill_(float("nan"))
        out.update(q_rot=q_rot, k_rot=k_rot, po=po, plse=plse, scaled=scaled, o=o, lse=lse, total=total)

    def look():
        _ok()
        now = [600, 18, 1, 321]
        _check_decode(out["q_rot"], kc, vc, rows, now, d ** -0.5, out["o"], out["lse"])
        _near_bf16(out["k_rot"], _turn64(src["k"], torch.tensor(now, device="cuda") - 1, 10000.0, 1.0), 1.2e-5)
        want, want_lse, mean_abs = _prompt64(out["q_rot"], out["k_rot"], src["v"], cu, d ** -0.5)
        _near_bf16(out["po"], want, (BF16_STEP + 1e-5) * mean_abs)
        assert float((out["plse"].double() - want_lse).abs().max()) <= 2e-5
        assert torch.equal(out["scaled"], out["po"].float() * 2) and torch.equal(out["total"], out["o"].float().sum(-1))

    for _ in range(3):
        steps()
    look()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for _ in range(5):
        for x in ("q_rot", "k_rot", "po", "plse", "o", "lse"):
            out[x].fill_(7.0)
        graph.replay()
        graph.replay()
        look()


# ------------------------------------------------------------------------------------------
# the largest sizes
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("n", [1 << 20, (1 << 27) + 5, (1 << 31) - 200])
@pytest.mark.parametrize("hq", [1, 9])
def test_decode_of_lengths_up_to_the_limit(n, hq):
    """A table whose entries all name one page, so that the tokens repeat: the result is that of the repeated
    tokens, each with its count, at any length that the table can hold."""
    d = 64
    # the largest pages with which the table stays within the library's limit of 2^31 - 129 tokens
    page = next(x for x in range(1 << 20, 0, -1) if -(-n // x) * x <= (1 << 31) - 129)
    width = -(-n // page)
    kc, vc = _randn(1, 2, page, 1, d), _randn(2, 2, page, 1, d)
    q = _randn(3, 2, hq, d)
    table = torch.ones(2, width, dtype=torch.int32, device="cuda")
    lens = [n, 3]
    o, lse = s2.decode(q, kc, vc, table, _ints(lens))
    _ok()
    # token t of the page is seen n // page times, those before n % page once more
    for b, m in enumerate(lens):
        count = torch.full((page,), m // page, dtype=torch.float64, device="cuda")
        count[:m % page] += 1
        k, v = kc[1, :, 0].double(), vc[1, :, 0].double()
        for h in range(hq):
            s = (k @ q[b, h].double()) * d ** -0.5
            want_lse = torch.logsumexp(s + count.log(), 0)
            p = torch.exp(s - want_lse) * count
            # fp32 sums of up to 2^31 terms: in 16-token steps, joined over 8 warps of 148 CTAs; one chain adds at
            # most 2^31 / (1184 * 16) = 2^16.8 terms, each off by 2^-24 of the sum, in random directions and at
            # worst all in one: 2^-7.2 of the weights' sum, o and l alike
            chain = m / (1184 * 16) * 2.0 ** -24
            _near_bf16(o[b, h], p @ v, (BF16_STEP + 1e-5 + 2 * chain) * (p @ v.abs()))
            assert abs(float(lse[b, h]) - float(want_lse)) <= 2e-5 + chain


def test_append_at_positions_up_to_the_limit():
    d, page, hkv = 64, 1 << 16, 1
    kc, vc = _randn(1, 2, page, hkv, d), _randn(2, 2, page, hkv, d)
    width = ((1 << 31) - 129) // page
    pos = [width * page - 1, width * page - 2, (1 << 30) + 12345]
    table = torch.zeros(3, width, dtype=torch.int32, device="cuda")
    k, v = _randn(3, 3, hkv, d), _randn(4, 3, hkv, d)
    _, k_rot = s2.rope_append(None, k, v, kc, vc, table, _ints([p + 1 for p in pos]), pi_scale=0.3)
    _ok()
    # (angles of 2^29 rad in 64 bits are good to 2^-23 rad; the kernel's to 1e-6)
    _near_bf16(k_rot, _turn64(k, torch.tensor(pos, device="cuda"), 10000.0, 0.3), 2.4e-5)
    for i, p in enumerate(pos):
        assert torch.equal(kc[0, p % page], k_rot[i]) and torch.equal(vc[0, p % page], v[i])
    # one token more than the table holds
    s2.rope_append(None, k, v, kc, vc, table, _ints([width * page + 1, 1, 1]))
    torch.cuda.synchronize()
    assert s2.s2attn_get_device_error() == (s2.S2ATTN_ERR_INVALID_ARG, (6 << 8) | 0x81)


@pytest.mark.parametrize("hq,hkv,lens", [
    (2, 1, [270000, 700]),                             # more than 2048 tiles of 128 rows: two launches
    (1, 1, [300, 530000]),                             # ... of 256 rows
    (1, 1, [139] * 60000 + [1]),                       # 8.3 million rows, 118 launches
])
def test_prompts_of_more_tiles_than_a_launch_takes(hq, hkv, lens):
    d = 64
    cu = _cu(lens)
    T = cu[-1]
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn(T, h, d, generator=g, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    o, lse = s2.prompt_fwd(q, k, v, torch.tensor(cu, dtype=torch.int32))
    _ok()
    assert o.isfinite().all() and lse.isfinite().all()
    r = random.Random(7)
    seqs = sorted({0, len(lens) - 1, len(lens) // 2} | {r.randrange(len(lens)) for _ in range(20)})
    for s in seqs:
        a, n = cu[s], lens[s]
        for i in sorted({0, n - 1, n // 2, r.randrange(n), max(0, n - 129)}):
            for h in range(hq):
                kk, vv = k[a:a + i + 1, h * hkv // hq].double(), v[a:a + i + 1, h * hkv // hq].double()
                sc = (kk @ q[a + i, h].double()) * d ** -0.5
                want = torch.logsumexp(sc, 0)
                p = torch.exp(sc - want)
                _near_bf16(o[a + i, h], p @ vv, (BF16_STEP + 1e-5) * (p @ vv.abs()))
                assert abs(float(lse[h, a + i]) - float(want)) <= 2e-5
