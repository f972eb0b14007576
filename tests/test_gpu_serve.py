"""The serving operators on the GPU: rotation and append to a paged cache, and decode over it,
against their definitions in 64 bits.

Tolerances. A bf16 output is the kernel's fp32 value rounded once, off by at most half a step,
2^-8 relative; the fp32 value itself differs from the exact one by
* append: the sine's and cosine's fp32 errors (angle to 2^-25 turns = 2e-7 rad, sincospif to a few
  2^-24) times |x|, so below 1e-6 (|x| + |y|);
* attention: P rounded to bf16 for the product (2^-8 relative each, at most 2^-8 sum p |v| / sum p
  <= 2^-8 max |v|), everything else in fp32 (below 1e-5 of the same). The bound used is
  2^-8 |o| + (2^-8 + 1e-5) * (sum p |v| / sum p), element by element.
LSE: fp32, scores of magnitude up to 2^5 or so: products summed in fp32 (128 terms, 2^-24 relative
to sum |q k| <= 40 |s|-ish terms) and log2/exp2 approximations of 2^-22: 2e-5 absolute covers them.
"""
import random

import pytest
import torch

import shifted_sparse_attention_fwd_b200 as s2

pytestmark = pytest.mark.gpu

BF16_STEP = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    s2.lib()


def _ok():
    torch.cuda.synchronize()
    st, code = s2.s2attn_get_device_error()
    assert st == s2.S2ATTN_OK, (st, hex(code))


def _randn(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _table(lens, page, seed, spare=2):
    """Random pages for sequences of `lens` tokens; unused entries hold a number far outside."""
    need = [-(-n // page) for n in lens]
    order = list(range(sum(need) + spare))
    random.Random(seed).shuffle(order)
    width, rows, at = max(1, max(need)), [], 0
    for n in need:
        rows.append(order[at:at + n] + [1 << 30] * (width - n))
        at += n
    return rows, len(order)


def _turn64(x, pos, base, pi):
    d = x.shape[-1]
    th = torch.tensor([base ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64, device=x.device)
    a = (pos.double()[:, None] * pi * th)[:, None]
    lo, hi = x[..., :d // 2].double(), x[..., d // 2:].double()
    return torch.cat((lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()), -1)


def _near_bf16(got, want, slack):
    """|got - want| <= half a bf16 step of the value, plus `slack`."""
    bad = (got.double() - want).abs() - (BF16_STEP * torch.maximum(got.double().abs(), want.abs()) + slack)
    assert got.isfinite().all() and float(bad.max()) <= 0, float(bad.max())


def _caches(seed, pages, page, hkv, d, layout):
    if layout == "kv_by_page":       # [pages, 2, page, Hkv, d]
        both = _randn(seed, pages, 2, page, hkv, d)
        return both[:, 0], both[:, 1]
    if layout == "kv_by_token":      # [pages, page, 2, Hkv, d]
        both = _randn(seed, pages, page, 2, hkv, d)
        return both[:, :, 0], both[:, :, 1]
    return _randn(seed, pages, page, hkv, d), _randn(seed + 1, pages, page, hkv, d)


# ------------------------------------------------------------------------------------------
# rotation and append
# ------------------------------------------------------------------------------------------
APPEND = [
    # new tokens, tokens before them, Hq, Hkv, d, page, pi_scale, layout
    ([1], [0], 4, 4, 64, 1, 1.0, "apart"),
    ([1, 1, 1], [0, 16, 4095], 8, 2, 128, 16, 0.5, "apart"),
    ([5, 0, 1, 0, 0, 77], [0, 3, 100, 0, 9, 31], 6, 2, 128, 24, 0.25, "kv_by_page"),
    ([9, 300, 8], [7, 1, 0], 5, 5, 64, 7, 1.0, "kv_by_token"),
    ([3] * 40, list(range(40)), 2, 1, 64, 48, 1.0, "apart"),
    ([2], [(1 << 24) - 40], 2, 2, 128, 1 << 16, 0.125, "apart"),      # a far position
]


@pytest.mark.parametrize("new,before,hq,hkv,d,page,pi,layout", APPEND)
@pytest.mark.parametrize("in_place", [False, True])
def test_append_matches_formula(new, before, hq, hkv, d, page, pi, layout, in_place):
    lens = [a + b for a, b in zip(new, before)]
    if max(lens) >= 1 << 20:
        # one huge virtual page table, all but the touched pages pointing at page 0
        rows, pages = [[0] * (max(lens) // page) + [1]], 2
        page_alloc = page
    else:
        rows, pages = _table(lens, page, 3)
        page_alloc = page
    T, behind = sum(new), 3
    q, k, v = (_randn(11 + i, T + behind, h, d) for i, h in enumerate((hq, hkv, hkv)))
    kc, vc = _caches(20, pages, page_alloc, hkv, d, layout)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q_in, k_in, kc0, vc0 = q.clone(), k.clone(), kc.clone(), vc.clone()
    q_rot = q if in_place else torch.full_like(q, 7.0)
    k_rot = k if in_place else torch.full_like(k, 7.0)
    s2.s2attn_rope_append(q, q_rot, k, k_rot, v, kc, vc, _ints(rows), _ints(lens), _ints(cu), pi_scale=pi)
    _ok()
    pos = torch.tensor([b + i for n, b in zip(new, before) for i in range(n)], device="cuda")
    want_q, want_k = _turn64(q_in[:T], pos, 10000.0, pi), _turn64(k_in[:T], pos, 10000.0, pi)
    slack = 1e-6 * 12                            # |x| + |y| below 12
    _near_bf16(q_rot[:T], want_q, slack)
    _near_bf16(k_rot[:T], want_k, slack)
    # rows behind the last sequence stay as they were
    assert torch.equal(q_rot[T:], q_in[T:] if in_place else torch.full_like(q_in[T:], 7.0))
    assert torch.equal(k_rot[T:], k_in[T:] if in_place else torch.full_like(k_in[T:], 7.0))
    # the cache: exactly these slots, with exactly these rows
    seq = torch.tensor([s for s, n in enumerate(new) for _ in range(n)], device="cuda")
    pg = torch.tensor(rows, device="cuda")[seq, pos // page]
    kc0[pg, pos % page] = k_rot[:T]
    vc0[pg, pos % page] = v[:T]
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)


def test_append_token_form_idle_rows_and_no_queries():
    lens, page, hkv, d = [5, 0, 33, 1], 8, 2, 64
    rows, pages = _table(lens, page, 1)
    k, v = _randn(1, 4, hkv, d), _randn(2, 4, hkv, d)
    kc, vc = _randn(3, pages, page, hkv, d), _randn(4, pages, page, hkv, d)
    kc0, vc0 = kc.clone(), vc.clone()
    s2.s2attn_rope_append(None, None, k, None, v, kc, vc, _ints(rows), _ints(lens))
    _ok()
    for s in (0, 2, 3):
        p = lens[s] - 1
        want = _turn64(k[s:s + 1], torch.tensor([p], device="cuda"), 10000.0, 1.0)[0]
        _near_bf16(kc[rows[s][p // page], p % page], want, 1.2e-5)
        kc0[rows[s][p // page], p % page] = kc[rows[s][p // page], p % page]
        vc0[rows[s][p // page], p % page] = v[s]
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)


def test_append_bad_page_and_length_are_reported_and_skipped():
    page, hkv, d = 8, 2, 64
    for table, lens, site in (([[0], [5]], [3, 3], 0x80), ([[0], [-1]], [3, 3], 0x80), ([[0], [1]], [3, 9], 0x81)):
        k, v = _randn(1, 2, hkv, d), _randn(2, 2, hkv, d)
        kc, vc = _randn(3, 2, page, hkv, d), _randn(4, 2, page, hkv, d)
        kc0, vc0 = kc.clone(), vc.clone()
        s2.s2attn_rope_append(None, None, k, None, v, kc, vc, _ints(table), _ints(lens))
        torch.cuda.synchronize()
        assert s2.s2attn_get_device_error() == (s2.S2ATTN_ERR_INVALID_ARG, (6 << 8) | site)
        assert s2.s2attn_get_device_error() == (s2.S2ATTN_OK, 0)
        kc0[0, 2], vc0[0, 2] = kc[0, 2], v[0]    # the good row's slot
        assert torch.equal(kc, kc0) and torch.equal(vc, vc0)


@pytest.mark.parametrize("hq,hkv,d,T", [(2, 1, 128, 5000), (4, 4, 64, 6001), (1, 1, 64, 4736), (9, 3, 64, 3001)])
def test_append_many_tokens_of_few_heads(hq, hkv, d, T):
    """Blocks of several groups of tokens, on views of one packed projection, ragged sequences, some of
    them empty; rows behind the last sequence untouched."""
    r = random.Random(T)
    new = [0]
    while sum(new) < T - 200:
        new.append(min(r.choice([0, 1, 31, 32, 33, 700]), T - sum(new)))
    T0, page = sum(new), 40
    rows, pages = _table(new, page, 4)
    packed = _randn(8, T, hq + 2 * hkv, d)
    q, k, v = packed[:, :hq], packed[:, hq:hq + hkv], packed[:, hq + hkv:]
    kc, vc = _caches(20, pages, page, hkv, d, "kv_by_token")
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    before = packed.clone()
    s2.s2attn_rope_append(q, q, k, k, v, kc, vc, _ints(rows), _ints(new), _ints(cu), pi_scale=0.5)
    _ok()
    pos = torch.tensor([i for n in new for i in range(n)], device="cuda")
    seq = torch.tensor([s for s, n in enumerate(new) for _ in range(n)], device="cuda")
    _near_bf16(packed[:T0, :hq + hkv], _turn64(before[:T0, :hq + hkv], pos, 10000.0, 0.5), 1.2e-5)
    assert torch.equal(packed[T0:], before[T0:]) and torch.equal(v, before[:, hq + hkv:])
    pg = torch.tensor(rows, device="cuda")[seq, pos // page]
    assert torch.equal(kc[pg, pos % page], k[:T0]) and torch.equal(vc[pg, pos % page], v[:T0])


# ------------------------------------------------------------------------------------------
# decode
# ------------------------------------------------------------------------------------------
def _decode64(q, kc, vc, rows, lens, scale):
    B, hq, d = q.shape
    page, hkv = kc.shape[1:3]
    g = hq // hkv
    o = torch.zeros(B, hq, d, dtype=torch.float64, device="cuda")
    mean_abs = torch.zeros_like(o)
    lse = torch.full((B, hq), float("-inf"), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        t = torch.arange(n, device="cuda")
        pg = torch.tensor(rows[b], device="cuda")[t // page]
        k, v = kc[pg, t % page].double(), vc[pg, t % page].double()
        for h in range(hq):
            s = (k[:, h // g] @ q[b, h].double()) * scale
            lse[b, h] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[b, h])
            o[b, h] = p @ v[:, h // g]
            mean_abs[b, h] = p @ v[:, h // g].abs()
    return o, lse, mean_abs


def _check_decode(q, kc, vc, rows, lens, scale, o, lse):
    want, want_lse, mean_abs = _decode64(q, kc, vc, rows, lens, scale)
    _near_bf16(o, want, (BF16_STEP + 1e-5) * mean_abs)
    empty = torch.tensor([n == 0 for n in lens], device="cuda")
    assert (lse[empty] == float("-inf")).all() and (o[empty] == 0).all()
    if not empty.all():
        assert float((lse[~empty].double() - want_lse[~empty]).abs().max()) <= 2e-5


DECODE = [
    # lens, Hq, Hkv, d, page, layout
    ([1], 1, 1, 64, 1, "apart"),
    ([1, 2, 15, 16, 17, 31, 33], 4, 4, 128, 16, "apart"),
    ([0, 130, 0, 0, 5], 8, 2, 64, 48, "kv_by_page"),
    ([700, 1, 4097], 6, 2, 128, 24, "kv_by_token"),
    ([513, 100], 16, 1, 128, 7, "apart"),          # a group of 16
    ([300, 45], 17, 1, 64, 32, "apart"),           # a group over one MMA's rows, odd
    ([90, 0, 1000], 40, 1, 128, 128, "apart"),     # three chunks of a group
    ([9000], 64, 8, 128, 64, "apart"),             # one long sequence, split over every SM
    ([33] * 300 + [0, 2000], 4, 4, 64, 16, "apart"),   # more sequences than a block has threads
    ([0, 0], 4, 2, 64, 16, "apart"),
    ([5000, 20000], 8, 8, 128, 64, "apart"),       # segments across warps and CTAs, one row each
    ([12000], 24, 2, 64, 16, "apart"),             # 12 rows: partials of 16-row warps
    ([47] * 40 + [4000], 8, 1, 128, 16, "apart"),
    ([500, 0, 77, 511, 16], 40, 2, 64, 32, "apart"),   # whole segments: 512 tokens at most, chunks of a group
    ([300] * 37, 4, 4, 128, 100, "kv_by_page"),    # ... one for each of 148 CTAs
    ([300] * 38, 4, 4, 128, 100, "kv_by_page"),    # ... and one sequence too many for that
]


@pytest.mark.parametrize("lens,hq,hkv,d,page,layout", DECODE)
def test_decode_matches_formula(lens, hq, hkv, d, page, layout):
    rows, pages = _table(lens, page, 5)
    kc, vc = _caches(30, pages, page, hkv, d, layout)
    q = _randn(33, len(lens), hq, d) * 2
    # what lies in the cache's other rows is never used
    used = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        if n:
            used[torch.tensor(rows[b], device="cuda")[t // page], t % page] = True
    for i, x in enumerate((kc, vc)):
        bad = torch.full((1,), float("nan") if i else float("inf"), device="cuda", dtype=x.dtype)
        x[~used] = bad
    o, lse = s2.decode(q, kc, vc, _ints(rows), _ints(lens))
    _ok()
    _check_decode(q, kc, vc, rows, lens, d ** -0.5, o, lse)
    o2, lse2 = s2.decode(q, kc, vc, _ints(rows), _ints(lens))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_bad_pages_and_lengths():
    """A page outside the cache counts as zeros, a length is cut to the table: reported, not followed."""
    page, hq, hkv, d = 16, 4, 2, 64
    q, kc, vc = _randn(1, 2, hq, d), _randn(2, 4, page, hkv, d), _randn(3, 4, page, hkv, d)
    for table, lens, site in (([[0, 1], [2, 4]], [20, 20], 0x80), ([[0, 1], [2, -7]], [20, 20], 0x80),
                              ([[0, 1], [2, 3]], [20, 33], 0x81), ([[0, 1], [2, 3]], [20, -1], 0x81)):
        o, lse = s2.decode(q, kc, vc, _ints(table), _ints(lens))
        torch.cuda.synchronize()
        assert s2.s2attn_get_device_error() == (s2.S2ATTN_ERR_INVALID_ARG, (7 << 8) | site)
        good_o, good_lse = s2.decode(q[:1], kc, vc, _ints(table[:1]), _ints(lens[:1]))
        _ok()
        assert torch.equal(lse[0], good_lse[0]) or float((lse[0] - good_lse[0]).abs().max()) < 1e-5


def test_decode_on_another_stream_and_in_a_graph():
    """A captured step follows the lengths and the tables of each replay."""
    page, hq, hkv, d, B = 16, 8, 2, 128, 3
    lens_list = [[40, 0, 1], [0, 333, 18], [512, 511, 513]]
    kc, vc = _randn(2, 99, page, hkv, d), _randn(3, 99, page, hkv, d)
    q = _randn(1, B, hq, d)
    lens = _ints([1] * B)
    table = torch.zeros(B, 33, dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(B, hq, device="cuda")
    ws = torch.empty(s2.s2attn_decode_workspace_size(B, hq, hkv, d), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s2.s2attn_decode(q, kc, vc, table, lens, o, lse, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s2.s2attn_decode(q, kc, vc, table, lens, o, lse, workspace=ws)
    for i, ll in enumerate(lens_list):
        rows, _ = _table(ll, page, i, spare=0)
        full = [r[:33] + [1 << 30] * (33 - len(r)) for r in rows]
        lens.copy_(_ints(ll))
        table.copy_(_ints(full))
        graph.replay()
        _ok()
        _check_decode(q, kc, vc, full, ll, d ** -0.5, o, lse)


def test_append_then_decode_as_a_model_answers():
    """Prompts appended, then three tokens appended and attended one by one, against attention in
    64 bits over the rotated rows."""
    hq, hkv, d, page, pi = 8, 2, 128, 16, 0.25
    prompts, steps = [37, 1, 200], 3
    lens = [n + steps for n in prompts]
    rows, pages = _table(lens, page, 9)
    table = _ints(rows)
    kc, vc = torch.zeros(pages, page, hkv, d, dtype=torch.bfloat16, device="cuda"), \
        torch.zeros(pages, page, hkv, d, dtype=torch.bfloat16, device="cuda")
    cu = [0, 37, 38, 238]
    q, k, v = (_randn(50 + i, 238, h, d) for i, h in enumerate((hq, hkv, hkv)))
    _, k_rot = s2.rope_append(q, k, v, kc, vc, table, _ints(prompts), _ints(cu), pi_scale=pi)
    keys = [[k_rot[cu[b]:cu[b + 1]]] for b in range(3)]
    vals = [[v[cu[b]:cu[b + 1]]] for b in range(3)]
    for step in range(steps):
        now = [n + step + 1 for n in prompts]
        q, k, v = (_randn(60 + 3 * step + i, 3, h, d) for i, h in enumerate((hq, hkv, hkv)))
        q_rot, k_rot = s2.rope_append(q, k, v, kc, vc, table, _ints(now), pi_scale=pi)
        o, lse = s2.decode(q_rot, kc, vc, table, _ints(now))
        _ok()
        _near_bf16(q_rot, _turn64(q, torch.tensor(now, device="cuda") - 1, 10000.0, pi), 1.2e-5)
        for b in range(3):
            keys[b].append(k_rot[b:b + 1])
            vals[b].append(v[b:b + 1])
            kk, vv = torch.cat(keys[b]).double(), torch.cat(vals[b]).double()
            assert kk.shape[0] == now[b]
            for h in range(hq):
                s = (kk[:, h // 4] @ q_rot[b, h].double()) * d ** -0.5
                p = torch.softmax(s, 0)
                _near_bf16(o[b, h], p @ vv[:, h // 4], (BF16_STEP + 1e-5) * (p @ vv[:, h // 4].abs()))
                assert abs(float(lse[b, h]) - float(torch.logsumexp(s, 0))) <= 2e-5


# ------------------------------------------------------------------------------------------
# prompts
# ------------------------------------------------------------------------------------------
def _prompt64(q, k, v, cu, scale):
    """o, lse and sum p |v| / sum p in 64 bits, sequence by sequence."""
    T, hq, d = q.shape
    g = hq // k.shape[1]
    o = torch.zeros(T, hq, d, dtype=torch.float64, device="cuda")
    mean_abs, lse = torch.zeros_like(o), torch.zeros(hq, T, dtype=torch.float64, device="cuda")
    for a, e in zip(cu, cu[1:]):
        mask = torch.ones(e - a, e - a, dtype=torch.bool, device="cuda").triu(1)
        for h in range(hq if e > a else 0):
            s = (q[a:e, h].double() @ k[a:e, h // g].double().T) * scale
            s = s.masked_fill(mask, float("-inf"))
            lse[h, a:e] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[h, a:e, None])
            vv = v[a:e, h // g].double()
            o[a:e, h], mean_abs[a:e, h] = p @ vv, p @ vv.abs()
    return o, lse, mean_abs


def _cu(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


PROMPT = [
    # lens, Hq, Hkv, d, rows before the first sequence, rows behind the last
    ([1], 1, 1, 64, 0, 0),
    ([113], 4, 4, 64, 0, 0),
    ([128], 2, 2, 128, 0, 0),
    ([129], 2, 2, 128, 0, 0),
    ([256, 257], 3, 3, 128, 0, 0),
    ([5, 127, 128, 0, 1, 300, 0, 17], 4, 2, 128, 3, 9),
    ([700, 8, 641], 8, 1, 64, 0, 130),
    ([1000, 385], 6, 2, 128, 1, 0),                # an odd group: 256 rows of one head
    ([2100], 2, 1, 128, 0, 0),
    ([2500, 31], 1, 1, 64, 0, 1),
    ([3] * 600 + [150], 2, 2, 64, 0, 0),           # more sequences than one launch takes
    ([640] * 9, 16, 8, 128, 0, 5),                 # more units than SMs: blocks taken over
]


@pytest.mark.parametrize("lens,hq,hkv,d,before,behind", PROMPT)
@pytest.mark.parametrize("packed", [False, True])
def test_prompt_matches_formula(lens, hq, hkv, d, before, behind, packed):
    cu = _cu(lens, before)
    T = cu[-1] + behind
    if packed:
        qkv = _randn(T, T, hq + 2 * hkv, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = (_randn(T + i, T, h, d) for i, h in enumerate((hq, hkv, hkv)))
    q *= 2
    # rows of no sequence hold anything and are left alone
    for t in (q, k, v):
        t[:before] = float("nan")
        t[cu[-1]:] = float("inf")
    o = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((hq, T), 7.0, device="cuda")
    s2.s2attn_prompt_fwd(q, k, v, o, lse, cu)
    _ok()
    want, want_lse, mean_abs = _prompt64(q, k, v, cu, d ** -0.5)
    a, e = cu[0], cu[-1]
    _near_bf16(o[a:e], want[a:e], (BF16_STEP + 1e-5) * mean_abs[a:e])
    assert float((lse[:, a:e].double() - want_lse[:, a:e]).abs().max()) <= 2e-5
    assert (o[:a] == 7).all() and (o[e:] == 7).all() and (lse[:, :a] == 7).all() and (lse[:, e:] == 7).all()
    o2, lse2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    s2.s2attn_prompt_fwd(q, k, v, o2, lse2, torch.tensor(cu, dtype=torch.int32))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (2, 2, 64)])
def test_prompt_growing_scores_and_other_sequences(hq, hkv, d):
    """Scores that grow along the keys by far more than 2^8 (the running maximum is rescaled again and
    again), next to sequences that hold NaN and infinities."""
    lens = [300, 777, 129, 60]
    cu = _cu(lens)
    q, k, v = (_randn(40 + i, cu[-1], h, d) for i, h in enumerate((hq, hkv, hkv)))
    q[cu[1]:cu[2]] = q[cu[1]:cu[2]].abs()
    ramp = torch.linspace(0, 12, lens[1], device="cuda")[:, None, None]
    k[cu[1]:cu[2]] = (k[cu[1]:cu[2]].float() * 0.1 + ramp).to(torch.bfloat16)
    for t, x in ((q, "nan"), (k, "inf"), (v, "nan")):
        t[cu[0]:cu[1]] = float(x)
        t[cu[2]:cu[3]] = float(x)
    o, lse = s2.prompt_fwd(q, k, v, cu, scale=0.5)
    _ok()
    for i in (1, 3):
        a, e = cu[i], cu[i + 1]
        want, want_lse, mean_abs = _prompt64(q[a:e], k[a:e], v[a:e], [0, e - a], 0.5)
        # scores reach 10^3 here, held to 24 bits: products of fp32 sums, 2^-20 relative and 1e-3
        # absolute in the exponent, which moves the weights by as much
        big = max(1.0, float(want_lse.abs().max()))
        _near_bf16(o[a:e], want, (BF16_STEP + 1e-5 + 2 * big * 2 ** -20) * mean_abs)
        assert float((lse[:, a:e].double() - want_lse).abs().max()) <= 2e-5 + big * 2 ** -20


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (3, 3, 64), (2, 2, 128)])
def test_prompt_values_of_hidden_rows(hq, hkv, d):
    """Keys and values that a row does not see never reach it, whatever they hold: rows before a row of NaN
    or infinities are what they were, to the bit, rows that see it are as the formula has them."""
    lens = [700, 130, 64, 257]
    cu = _cu(lens)
    q, k, v = (_randn(45 + i, cu[-1], h, d) for i, h in enumerate((hq, hkv, hkv)))
    want, want_lse = s2.prompt_fwd(q, k, v, cu)
    # (sequence, row, column, value)
    bad = [(0, 0, 5, "nan"), (0, 255, 0, "inf"), (0, 256, 0, "-inf"), (0, 640, 9, "-inf"), (0, 699, d - 1, "nan"),
           (1, 129, 33, "inf"), (2, 13, 7, "inf"), (2, 40, 7, "inf"), (3, 127, 1, "nan"), (3, 128, 2, "inf"), (3, 256, 3, "-inf")]
    sign = torch.zeros(cu[-1], hkv, d, dtype=torch.float64, device="cuda")   # running sum of what is seen
    for s_, r, c, x in bad:
        h = (r + c) % hkv
        v[cu[s_] + r, h, c] = float(x)
        sign[cu[s_] + r:cu[s_ + 1], h, c] += float(x)
    o, lse = s2.prompt_fwd(q, k, v, cu)
    _ok()
    assert torch.equal(lse, want_lse)
    seen = sign.repeat_interleave(hq // hkv, 1)
    clean = seen == 0
    # a unit that holds such a value has zeros in its place, so nothing else may move
    assert torch.equal(o[clean], want[clean])
    got = o.double()
    assert torch.equal(got[seen.isinf()], seen[seen.isinf()]) and got[seen.isnan()].isnan().all()
    # keys: the rows behind a key of NaN have NaN, those before it are untouched
    k[cu[1] + 100, 0, 3] = float("nan")
    o2, lse2 = s2.prompt_fwd(q, k, v, cu)
    _ok()
    g = hq // hkv
    rows = slice(cu[1] + 100, cu[2])
    assert o2[rows, :g].isnan().all() and lse2[:g, rows].isnan().all()
    keep = torch.ones(cu[-1], hq, dtype=torch.bool, device="cuda")
    keep[rows, :g] = False
    same = (o2 == o) | (o2.isnan() & o.isnan())
    assert same[keep].all() and torch.equal(lse2[keep.T], lse[keep.T])


@pytest.mark.parametrize("hq,hkv,d", [(3, 3, 128), (9, 3, 64), (4, 2, 128)])
def test_prompts_of_a_few_tokens_by_the_hundred(hq, hkv, d):
    """Units of one query tile and of two, many for each CTA, in any order: right, and the values that a row
    does not see (of its own sequence, and of the neighbour that shares its tile of values) never reach it."""
    lens = [40, 128, 1, 130, 256, 300, 7, 390, 16, 127, 64, 129] * 20
    cu = _cu(lens)
    q, k, v = (_randn(50 + i, cu[-1], h, d) for i, h in enumerate((hq, hkv, hkv)))
    o, lse = s2.prompt_fwd(q, k, v, cu)
    _ok()
    want, want_lse, mean_abs = _prompt64(q, k, v, cu, d ** -0.5)
    _near_bf16(o, want, (BF16_STEP + 1e-5) * mean_abs)
    assert float((lse.double() - want_lse).abs().max()) <= 2e-5
    sign = torch.zeros(cu[-1], hkv, d, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        for r, x in ((0, "inf"), (n - 1, "nan"), (n // 2, "-inf")) if i % 5 == 2 else ():
            v[cu[i] + r, (i + r) % hkv, (7 * i + r) % d] = float(x)
        a, e = cu[i], cu[i + 1]
        sign[a:e] = torch.where(v[a:e].isfinite(), torch.zeros_like(v[a:e]), v[a:e]).double().cumsum(0)
    o2, lse2 = s2.prompt_fwd(q, k, v, cu)
    _ok()
    assert torch.equal(lse2, lse)
    seen = sign.repeat_interleave(hq // hkv, 1)
    hit = ~(seen == 0)
    dirty = torch.zeros(cu[-1], dtype=torch.bool, device="cuda")
    for i in range(2, len(lens), 5):
        dirty[cu[i]:cu[i + 1]] = True
    assert torch.equal(o2[~dirty], o[~dirty])
    got = o2.double()
    assert got[~hit].isfinite().all()
    assert torch.equal(got[seen.isinf()], seen[seen.isinf()]) and got[seen.isnan()].isnan().all()


def test_prompt_append_decode_agree():
    """A prompt through append and prompt_fwd, then its last row again as a decoding step: the same
    attention from the cache."""
    hq, hkv, d, page = 8, 2, 128, 32
    lens = [200, 1, 513]
    cu = _cu(lens)
    rows, pages = _table(lens, page, 2)
    q, k, v = (_randn(70 + i, cu[-1], h, d) for i, h in enumerate((hq, hkv, hkv)))
    kc, vc = _randn(1, pages, page, hkv, d), _randn(2, pages, page, hkv, d)
    q_rot, k_rot = s2.rope_append(q, k, v, kc, vc, _ints(rows), _ints(lens), _ints(cu), pi_scale=0.5)
    o, lse = s2.prompt_fwd(q_rot, k_rot, v, cu)
    last = torch.tensor(cu[1:], device="cuda") - 1
    o1, lse1 = s2.decode(q_rot[last], kc, vc, _ints(rows), _ints(lens))
    _ok()
    want, want_lse, mean_abs = _prompt64(q_rot, k_rot, v, cu, d ** -0.5)
    slack = (BF16_STEP + 1e-5) * mean_abs
    _near_bf16(o, want, slack)
    _near_bf16(o1, want[last], slack[last])
    assert float((lse.double() - want_lse).abs().max()) <= 2e-5
    assert float((lse1.double() - want_lse[:, last].T).abs().max()) <= 2e-5


# ------------------------------------------------------------------------------------------
# large offsets, graphs, streams, shared pages
# ------------------------------------------------------------------------------------------
def test_offsets_past_32_bits():
    """Pages, rows and heads whose element offsets pass 2^31 and 2^32: caches of 33,000 pages of 64 x 8 x
    128, K and V interleaved by page, and packed rows 2^17 elements apart."""
    page, hkv, hq, d = 64, 8, 16, 128
    pages = 33000
    both = torch.empty(pages, 2, page, hkv, d, dtype=torch.bfloat16, device="cuda")   # 8.6 GB
    kc, vc = both[:, 0], both[:, 1]
    lens = [100, 64, 129]
    rows = [[32999, 16400, 1 << 30], [16383, 1 << 30, 1 << 30], [0, 32998, 16384]]
    cu = _cu(lens)
    T = cu[-1]
    q, k, v = (_randn(90 + i, T, h, d) for i, h in enumerate((hq, hkv, hkv)))
    q_rot, k_rot = s2.rope_append(q, k, v, kc, vc, _ints(rows), _ints(lens), _ints(cu))
    for s, n in enumerate(lens):
        for t in range(n):
            pg = rows[s][t // page]
            assert torch.equal(kc[pg, t % page], k_rot[cu[s] + t]) and torch.equal(vc[pg, t % page], v[cu[s] + t])
    last = torch.tensor(cu[1:], device="cuda") - 1
    o, lse = s2.decode(q_rot[last], kc, vc, _ints(rows), _ints(lens))
    _ok()
    want, want_lse, mean_abs = _prompt64(q_rot, k_rot, v, cu, d ** -0.5)
    _near_bf16(o, want[last], (BF16_STEP + 1e-5) * mean_abs[last])
    assert float((lse.double() - want_lse[:, last].T).abs().max()) <= 2e-5
    del both, kc, vc
    # packed rows far apart: row 20,000 of o, q is past 2^31 elements
    n, before = 300, 20000
    buf = torch.empty(before + n, 1 << 17, dtype=torch.bfloat16, device="cuda")   # 5.3 GB
    views = [buf[:, i * 4096:i * 4096 + h * d].unflatten(1, (h, d)) for i, h in enumerate((hq, hkv, hkv, hq))]
    for i, h in enumerate((hq, hkv, hkv)):
        views[i][before:] = _randn(95 + i, n, h, d)
    qv, kv, vv, ov = views
    lse = torch.empty(hq, before + n, device="cuda")
    s2.s2attn_prompt_fwd(qv, kv, vv, ov, lse, [before, before + n])
    _ok()
    want, want_lse, mean_abs = _prompt64(qv[before:], kv[before:], vv[before:], [0, n], d ** -0.5)
    _near_bf16(ov[before:], want, (BF16_STEP + 1e-5) * mean_abs)
    assert float((lse[:, before:].double() - want_lse).abs().max()) <= 2e-5


def test_captured_step_of_append_and_decode():
    """One decoding step captured through the allocating calls, replayed as the sequences grow; the second
    graph shares nothing with the first and both stay right when replayed in turn."""
    hq, hkv, d, page, B, pi = 8, 4, 64, 8, 3, 0.5
    width = 80                                       # 640 tokens: the list form, two launches
    order = list(range(B * width))
    random.Random(3).shuffle(order)
    rows = [order[b * width:(b + 1) * width] for b in range(B)]
    table = _ints(rows)
    graphs = []
    for g in range(2):
        kc, vc = _randn(5 + g, B * width, page, hkv, d), _randn(7 + g, B * width, page, hkv, d)
        st = dict(kc=kc, vc=vc, q=_randn(1, B, hq, d), k=_randn(2, B, hkv, d), v=_randn(3, B, hkv, d),
                  lens=_ints([3, 0, 40]), graph=torch.cuda.CUDAGraph())
        s2.rope_append(st["q"], st["k"], st["v"], kc.clone(), vc.clone(), table, st["lens"], pi_scale=pi)
        s2.decode(st["q"], kc, vc, table, st["lens"])
        torch.cuda.synchronize()
        with torch.cuda.graph(st["graph"]):
            st["q_rot"], st["k_rot"] = s2.rope_append(st["q"], st["k"], st["v"], kc, vc, table, st["lens"], pi_scale=pi)
            st["o"], st["lse"] = s2.decode(st["q_rot"], kc, vc, table, st["lens"])
        graphs.append(st)
    lens = [[200, 0, 40], [639, 1, 7]]
    for step in range(3):
        for g, st in enumerate(graphs):
            now = [n + 1 if n else 0 for n in lens[g]]
            lens[g] = [min(n, 640) for n in now]
            for x, h in (("q", hq), ("k", hkv), ("v", hkv)):
                st[x].copy_(_randn(100 + 10 * step + g, B, h, d))
            st["lens"].copy_(_ints(lens[g]))
            st["graph"].replay()
            _ok()
            for b, n in enumerate(lens[g]):
                if n:
                    want = _turn64(st["k"][b:b + 1], torch.tensor([n - 1], device="cuda"), 10000.0, pi)[0]
                    _near_bf16(st["kc"][rows[b][(n - 1) // page], (n - 1) % page], want, 1.2e-5)
            _check_decode(st["q_rot"], st["kc"], st["vc"], rows, lens[g], d ** -0.5, st["o"], st["lse"])


def test_captured_prompt_and_calls_on_a_side_stream():
    hq, hkv, d = 6, 3, 64
    cu = _cu([200, 1, 300])
    q, k, v = (_randn(i, cu[-1], h, d) for i, h in enumerate((hq, hkv, hkv)))
    o, lse = s2.prompt_fwd(q, k, v, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o1, lse1 = s2.prompt_fwd(q, k, v, cu, stream=side)
    o2, lse2 = s2.prompt_fwd(q, k, v, cu, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, lse3 = s2.prompt_fwd(q, k, v, cu)
    graph.replay()
    _ok()
    for x, y in ((o1, lse1), (o2, lse2), (o3, lse3)):
        assert torch.equal(x, o) and torch.equal(y, lse)
    q.copy_(_randn(9, cu[-1], hq, d))
    graph.replay()
    o4, lse4 = s2.prompt_fwd(q, k, v, cu)
    _ok()
    assert torch.equal(o3, o4) and torch.equal(lse3, lse4)


def test_two_calls_at_once_and_shared_pages():
    """Decoding steps on two streams at once, and sequences that share the pages of a common prefix."""
    hq, hkv, d, page = 16, 4, 128, 16
    prefix = list(range(40))                         # 640 tokens that all sequences share
    lens = [640 + n for n in (1, 17, 300, 0)]
    own = [[40], [41, 42], list(range(43, 62)), []]
    rows = [prefix + x + [1 << 30] * (19 - len(x)) for x in own]
    kc, vc = _randn(2, 62, page, hkv, d), _randn(3, 62, page, hkv, d)
    qs = [_randn(10 + i, 4, hq, d) for i in range(2)]
    want = [s2.decode(q, kc, vc, _ints(rows), _ints(lens)) for q in qs]
    for q, (o, lse) in zip(qs, want):
        _check_decode(q, kc, vc, rows, lens, d ** -0.5, o, lse)
    streams = [torch.cuda.Stream() for _ in qs]
    table, n = _ints(rows), _ints(lens)
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for q, s in zip(qs, streams):
            with torch.cuda.stream(s):
                got.append(s2.decode(q, kc, vc, table, n))
    _ok()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


def test_append_without_queries_and_views_of_length_one():
    hkv, d, page = 1, 64, 1
    kc, vc = _randn(1, 3, page, hkv, d), _randn(2, 3, page, hkv, d)
    big = _randn(3, 4, 5, d)
    k, v = big[1:2, 2:3], big[2:3, 4:5]              # one row, one head: strides of the packed rows
    q_rot, k_rot = s2.rope_append(None, k, v, kc, vc, _ints([[0, 2]]), _ints([2]))
    _ok()
    assert q_rot is None
    _near_bf16(k_rot, _turn64(k, torch.tensor([1], device="cuda"), 10000.0, 1.0), 1.2e-5)
    assert torch.equal(kc[2, 0], k_rot[0]) and torch.equal(vc[2, 0], v[0])
    with pytest.raises(s2.S2AttnError, match="invalid"):
        s2.decode(k, kc[:, :, :, :], vc, _ints([[0, 2]]), _ints([2]), scale=0.0)
    with pytest.raises(ValueError, match="contiguous"):
        s2.decode(big.transpose(1, 2)[:, :, :].reshape(4, 5, d).transpose(0, 1)[:, :, ::2], kc, vc, _ints([[0]] * 5), _ints([1] * 5))


def test_steps_in_a_row_without_a_wait():
    """Two hundred decoding steps queued one behind another, with no wait in between (each kernel may start
    before the one in front of it has ended): the cache and the last outputs are those of the formula."""
    hq, hkv, d, page, pi = 8, 2, 64, 16, 0.5
    start, steps = [600, 5, 0, 130], 200
    lens = [n + steps for n in start]
    rows, pages = _table(lens, page, 8)
    kc, vc = _randn(1, pages, page, hkv, d), _randn(2, pages, page, hkv, d)
    kc0, vc0 = kc.clone(), vc.clone()
    table, now = _ints(rows), _ints(start)
    q, k, v = (_randn(3 + i, steps * 4, h, d).view(steps, 4, h, d) for i, h in enumerate((hq, hkv, hkv)))
    outs = []
    for i in range(steps):
        now += 1
        q_rot, k_rot = s2.rope_append(q[i], k[i], v[i], kc, vc, table, now, pi_scale=pi)
        outs.append((q_rot, k_rot, *s2.decode(q_rot, kc, vc, table, now)))
    _ok()
    for b, n in enumerate(start):
        for i in range(steps):
            kc0[rows[b][(n + i) // page], (n + i) % page] = outs[i][1][b]
            vc0[rows[b][(n + i) // page], (n + i) % page] = v[i, b]
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)
    for i in (0, 1, 57, 199):
        q_rot, k_rot, o, lse = outs[i]
        seen = [n + i + 1 for n in start]
        _near_bf16(k_rot, _turn64(k[i], torch.tensor(seen, device="cuda") - 1, 10000.0, pi), 1.2e-5)
        _check_decode(q_rot, kc, vc, rows, seen, d ** -0.5, o, lse)


def test_decode_views_own_workspace_and_no_lse():
    """q and o as views of wider buffers, a workspace full of NaN used by one call after another, no lse."""
    hq, hkv, d, page = 12, 2, 128, 16
    lens = [900, 3, 0, 2048]
    rows, pages = _table(lens, page, 6)
    kc, vc = _caches(11, pages, page, hkv, d, "kv_by_page")
    packed, out = _randn(1, 4, 3 * hq, d), _randn(2, 4, 2 * hq, d)
    q, o = packed[:, hq:2 * hq], out[:, hq:]
    before = out.clone()
    ws = torch.full((s2.s2attn_decode_workspace_size(4, hq, hkv, d),), 255, dtype=torch.uint8, device="cuda")
    lse = torch.empty(4, hq, device="cuda")
    table, n = _ints(rows), _ints(lens)
    s2.s2attn_decode(q, kc, vc, table, n, o, lse, workspace=ws)
    _ok()
    _check_decode(q, kc, vc, rows, lens, d ** -0.5, o, lse)
    assert torch.equal(out[:, :hq], before[:, :hq])
    first = o.clone()
    o.zero_()
    s2.s2attn_decode(q, kc, vc, table, n, o, None, workspace=ws)
    _ok()
    assert torch.equal(o, first)
    with pytest.raises(s2.S2AttnError, match="invalid"):
        s2.s2attn_decode(q, kc, vc, table, n, o, None, workspace=ws[:-256])


def test_decode_of_thousands_of_sequences():
    r = random.Random(1)
    lens = [r.choice([0, 1, 15, 16, 17, 40]) for _ in range(3000)] + [3000]
    hq, hkv, d, page = 2, 1, 64, 8
    rows, pages = _table(lens, page, 2)
    kc, vc = _randn(1, pages, page, hkv, d), _randn(2, pages, page, hkv, d)
    q = _randn(3, len(lens), hq, d)
    o, lse = s2.decode(q, kc, vc, _ints(rows), _ints(lens))
    _ok()
    pick = [i for i in range(0, 3000, 61)] + [2999, 3000]
    at = torch.tensor(pick, device="cuda")
    _check_decode(q[at], kc, vc, [rows[i] for i in pick], [lens[i] for i in pick], d ** -0.5, o[at], lse[at])
    empty = torch.tensor([n == 0 for n in lens], device="cuda")
    assert (o[empty] == 0).all() and (lse[empty] == float("-inf")).all() and o.isfinite().all()


def test_prompts_of_no_rows():
    q = _randn(1, 7, 2, 64)
    o, lse = torch.full_like(q, 7.0), torch.full((2, 7), 7.0, device="cuda")
    for cu in ([0, 0], [3, 3, 3], [7, 7]):
        s2.s2attn_prompt_fwd(q, q, q, o, lse, cu)
    _ok()
    assert (o == 7).all() and (lse == 7).all()
