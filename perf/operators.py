"""The serving operators' cases: what each is measured on, its plain form and its exact values.

Three operators that a model fine-tuned with S²-Attn is served with (full attention, rotary
positions rescaled by Position Interpolation, a paged key/value cache):

* ``append``  keys and values of new tokens go into the paged cache, queries and keys turned by
              their rotary angle on the way (``rope_append``);
* ``decode``  attention of one new token per sequence over the paged cache (``decode``);
* ``prompt``  causal attention over packed prompts of different lengths (``prompt_fwd``).

With ``own`` false, ``run`` computes them from elementary torch operations in fp32 (angles in
fp64: positions reach 2^17 and more); with ``own`` true it calls the framework.
"""
import math
import random

import torch

own = False

BASE = 10000.0   # the frequency base of Llama 2


# ----------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------
def listed():
    return [
        # the next token of one short conversation: latency is all that counts
        dict(name="append_token_1", op="append", form="token", seqs=1, longest=700, even=False, heads=32,
             kv_heads=32, d=128, page=16, pi=1.0, lens_seed=1),
        # one step of a running batch, grouped heads, far positions of a 32k context
        dict(name="append_token_64_gqa", op="append", form="token", seqs=64, longest=4096, even=False,
             heads=64, kv_heads=8, d=128, page=64, pi=0.125, lens_seed=2),
        # a batch of prompts of very different lengths, small heads, pages that end inside a tile
        dict(name="append_prompts_d64", op="append", form="prompt", seqs=21, longest=3001, even=False,
             heads=4, kv_heads=4, d=64, page=48, pi=0.5, lens_seed=3),
        # one long prompt of a 32k context, grouped heads: bandwidth
        dict(name="append_prompt_32768_gqa", op="append", form="prompt", seqs=1, longest=32768, even=True,
             heads=64, kv_heads=8, d=128, page=64, pi=0.125, lens_seed=4),
        # one short sequence, small heads: latency
        dict(name="decode_1_short_d64", op="decode", seqs=1, longest=131, even=True, idle=False, heads=4,
             kv_heads=4, d=64, page=16, lens_seed=5),
        # a running batch of the 7B layer at an 8k context, every sequence about as long
        dict(name="decode_16_mha", op="decode", seqs=16, longest=8192, even=True, idle=False, heads=32,
             kv_heads=32, d=128, page=64, lens_seed=6),
        # a ragged batch of the 70B layer, up to a 32k context, with a padding row
        dict(name="decode_64_gqa_ragged", op="decode", seqs=64, longest=32768, even=False, idle=True,
             heads=64, kv_heads=8, d=128, page=32, lens_seed=7),
        # one sequence of a 100k context: the cache's length is the only axis to split
        dict(name="decode_1_long_gqa", op="decode", seqs=1, longest=102400, even=True, idle=False, heads=64,
             kv_heads=8, d=128, page=128, lens_seed=8),
        # one short prompt, small heads: latency
        dict(name="prompt_1_short_d64", op="prompt", seqs=1, longest=113, even=True, heads=4, kv_heads=4,
             d=64, lens_seed=9),
        # packed prompts of very different lengths, the 7B layer's heads
        dict(name="prompt_ragged_mha", op="prompt", seqs=12, longest=4999, even=False, heads=32, kv_heads=32,
             d=128, lens_seed=10),
        # one 8k prompt, the 7B layer's heads
        dict(name="prompt_8192_mha", op="prompt", seqs=1, longest=8192, even=True, heads=32, kv_heads=32,
             d=128, lens_seed=11),
        # two long prompts of the 70B layer
        dict(name="prompt_long_gqa", op="prompt", seqs=2, longest=20480, even=True, heads=64, kv_heads=8,
             d=128, lens_seed=12),
    ]


def lens_of(case):
    """The sequences' lengths: the first is the longest; the others within an eighth of it
    (`even`), or spread over the logarithm of the whole range; an idle row has length 0."""
    r = random.Random(case["lens_seed"])
    top = case["longest"]
    lens = [top]
    for _ in range(case["seqs"] - 1):
        lens.append(top - r.randrange(top // 8 + 1) if case["even"]
                    else max(1, min(top, round(math.exp(r.uniform(0.0, math.log(top)))))))
    if case.get("idle") and len(lens) > 1:
        lens[-1] = 0
    return lens


def _log(r, lo, hi):
    return max(lo, min(hi, round(math.exp(r.uniform(math.log(lo), math.log(hi))))))


HEADS = [(4, 4), (8, 2), (6, 2), (5, 1), (16, 16), (32, 32), (32, 8), (64, 8)]


def draw(rng):
    op = rng.choice(["append", "decode", "prompt"])
    heads, kv_heads = rng.choice(HEADS)
    d = rng.choice([64, 128, 128])
    page = rng.choice([8, 16, 24, 32, 48, 64, 128, 256])
    c = dict(op=op, heads=heads, kv_heads=kv_heads, d=d, lens_seed=rng.randrange(1 << 30))
    if op == "append":
        form = rng.choice(["token", "prompt"])
        seqs = _log(rng, 1, 64 if form == "token" else 24)
        c.update(form=form, page=page, pi=rng.choice([1.0, 0.5, 0.25, 0.125]), seqs=seqs, even=False,
                 longest=_log(rng, 8, 4096 if form == "token" else 16384 // seqs + 512))
    elif op == "decode":
        seqs = _log(rng, 1, 128)
        c.update(page=page, seqs=seqs, even=rng.random() < 0.5, idle=rng.random() < 0.5,
                 longest=_log(rng, 1, min(65536, 4_000_000 // (seqs * kv_heads))))
    else:
        seqs = _log(rng, 1, 24)
        c.update(seqs=seqs, even=rng.random() < 0.5, longest=_log(rng, 1, 12288 // seqs + 256))
    return c


# ----------------------------------------------------------------------------------------
# What a user's program has in hand
# ----------------------------------------------------------------------------------------
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cache(case, gen, seed, lens):
    """A page pool with the sequences' pages spread over it at random, and a few spare pages."""
    page = case["page"]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    order = list(range(pages))
    random.Random(seed).shuffle(order)
    width = max(1, max(need))
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    shape = (pages, page, case["kv_heads"], case["d"])
    return _randn(gen, *shape), _randn(gen, *shape), _ints(table)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens = lens_of(case)
    hq, hkv, d = case["heads"], case["kv_heads"], case["d"]
    s = dict(case=case)
    if case["op"] == "append":
        kc, vc, table = _cache(case, gen, seed, lens)
        new = [1] * len(lens) if case["form"] == "token" else lens
        t = sum(new)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s.update(q=_randn(gen, t, hq, d), k=_randn(gen, t, hkv, d), v=_randn(gen, t, hkv, d), k_cache=kc,
                 v_cache=vc, table=table, lens=_ints(lens), cu=_ints(cu))
    elif case["op"] == "decode":
        kc, vc, table = _cache(case, gen, seed, lens)
        s.update(q=_randn(gen, len(lens), hq, d), k_cache=kc, v_cache=vc, table=table, lens=_ints(lens),
                 scale=d ** -0.5)
    else:
        t = sum(lens)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        # the lengths of a batch of prompts are the scheduler's own numbers: they are on the host
        s.update(q=_randn(gen, t, hq, d), k=_randn(gen, t, hkv, d), v=_randn(gen, t, hkv, d),
                 cu=torch.tensor(cu, dtype=torch.int32), cu_dev=_ints(cu), scale=d ** -0.5)
    return s


# ----------------------------------------------------------------------------------------
# The plain forms
# ----------------------------------------------------------------------------------------
def _plain_append(s):
    q, k, v, table, lens, cu = s["q"], s["k"], s["v"], s["table"], s["lens"].long(), s["cu"].long()
    page, d = s["k_cache"].shape[1], q.shape[2]
    tok = torch.arange(q.shape[0], device=q.device)
    seq = torch.searchsorted(cu, tok, right=True) - 1
    pos = lens[seq] - (cu[seq + 1] - cu[seq]) + (tok - cu[seq])
    i = torch.arange(d // 2, device=q.device, dtype=torch.float64)
    ang = (pos.double() * s["case"]["pi"])[:, None] * torch.exp(-(2.0 * i / d) * math.log(BASE))
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]

    def turn(x):
        a, b = x[..., :d // 2].float(), x[..., d // 2:].float()
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1).to(torch.bfloat16)

    q_rot, k_rot = turn(q), turn(k)
    slot = table[seq, pos // page].long() * page + pos % page
    s["k_cache"].view(-1, *k.shape[1:])[slot] = k_rot
    s["v_cache"].view(-1, *v.shape[1:])[slot] = v
    return dict(q_rot=q_rot, k_rot=k_rot, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_decode(s):
    q, table, lens = s["q"], s["table"].long(), s["lens"].long()
    b, hq, d = q.shape
    page, hkv = s["k_cache"].shape[1:3]
    at = table.clamp(min=0)
    qf = q.float().view(b, hkv, hq // hkv, d) * s["scale"]
    k = s["k_cache"][at].view(b, -1, hkv, d).permute(0, 2, 3, 1).float()
    sc = qf @ k
    del k
    seen = torch.arange(sc.shape[3], device=q.device) < lens[:, None]
    sc.masked_fill_(~seen[:, None, None], float("-inf"))
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    v = s["v_cache"][at].view(b, -1, hkv, d).permute(0, 2, 1, 3).float()
    o = (p @ v) / torch.where(total == 0, torch.ones_like(total), total)
    return dict(o=o.view(b, hq, d).to(torch.bfloat16), lse=(m + torch.log(total)).view(b, hq))


def _plain_prompt(s):
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu_dev"].long()
    t, hq, d = q.shape
    hkv = k.shape[1]
    tok = torch.arange(t, device=q.device)
    first = cu[torch.searchsorted(cu, tok, right=True) - 1]
    hidden = (tok[None, :] > tok[:, None]) | (tok[None, :] < first[:, None])
    o, lse = torch.empty_like(q), torch.empty(hq, t, dtype=torch.float32, device=q.device)
    o4, lse4 = o.view(t, hkv, -1, d), lse.view(hkv, -1, t)
    step = max(1, (1 << 32) // (t * t * (hq // hkv)))
    for h in range(0, hkv, step):   # the scores of `step` key/value heads fit the memory at once
        qf = q.view(t, hkv, -1, d)[:, h:h + step].permute(1, 2, 0, 3).float() * s["scale"]
        kf, vf = (x[:, h:h + step].permute(1, 0, 2)[:, None].float() for x in (k, v))
        sc = qf @ kf.transpose(2, 3)
        sc.masked_fill_(hidden, float("-inf"))
        m = sc.amax(-1, keepdim=True)
        p = sc.sub_(m).exp_()
        total = p.sum(-1, keepdim=True)
        o4[:, h:h + step] = ((p @ vf) / total).permute(2, 0, 1, 3).to(torch.bfloat16)
        lse4[h:h + step] = (m + torch.log(total))[..., 0]
    return dict(o=o, lse=lse)


def run(state):
    op = state["case"]["op"]
    if own:
        import shifted_sparse_attention_fwd_b200 as s2
        if op == "append":
            q_rot, k_rot = s2.rope_append(state["q"], state["k"], state["v"], state["k_cache"],
                                          state["v_cache"], state["table"], state["lens"],
                                          cu_seqlens=None if state["case"]["form"] == "token" else state["cu"],
                                          base=BASE, pi_scale=state["case"]["pi"])
            return dict(q_rot=q_rot, k_rot=k_rot, k_cache=state["k_cache"], v_cache=state["v_cache"])
        if op == "decode":
            o, lse = s2.decode(state["q"], state["k_cache"], state["v_cache"], state["table"],
                               state["lens"], state["scale"])
        else:
            o, lse = s2.prompt_fwd(state["q"], state["k"], state["v"], state["cu"], state["scale"])
        return dict(o=o, lse=lse)
    return {"append": _plain_append, "decode": _plain_decode, "prompt": _plain_prompt}[op](state)


# ----------------------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------------------
def work(case):
    lens = lens_of(case)
    hq, hkv, d = case["heads"], case["kv_heads"], case["d"]
    if case["op"] == "append":
        t = len(lens) if case["form"] == "token" else sum(lens)
        # q, k, v read; turned q and k, and both caches' new rows written; 6 flops a turned pair
        return {"bytes": t * d * 2 * (2 * hq + 5 * hkv), "flops": 3 * t * d * (hq + hkv)}
    if case["op"] == "decode":
        t = sum(lens)
        return {"bytes": 2 * t * hkv * d * 2 + len(lens) * hq * (4 * d + 4), "flops": 4 * t * hq * d}
    t = sum(lens)
    return {"bytes": t * d * 2 * (2 * hq + 2 * hkv) + 4 * t * hq,
            "flops": 4 * d * hq * sum(n * (n + 1) // 2 for n in lens)}


# ----------------------------------------------------------------------------------------
# The definition in 64 bits, sequence by sequence
# ----------------------------------------------------------------------------------------
def _attend64(q, k, v, scale, first):
    """Rows of softmax(scale q k^T) v for one kv head, q [G, n, d] at positions first, first + 1, ..."""
    sc = torch.matmul(q, k.T) * scale
    n, m = sc.shape[1:]
    seen = torch.arange(m, device=q.device)[None] <= first + torch.arange(n, device=q.device)[:, None]
    sc = torch.where(seen, sc, torch.full((), -math.inf, dtype=torch.float64, device=q.device))
    lse = torch.logsumexp(sc, -1)
    return torch.matmul(torch.exp(sc - lse[..., None]), v), lse


def exact(case, seed):
    s = prepare(case, seed)
    lens = lens_of(case)
    hq, hkv, d = case["heads"], case["kv_heads"], case["d"]
    g = hq // hkv
    if case["op"] == "append":
        kc, vc, table = s["k_cache"].double(), s["v_cache"].double(), s["table"].tolist()
        theta = torch.tensor([BASE ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64, device="cuda")
        q_rot, k_rot, row = s["q"].double(), s["k"].double(), 0
        for b, n in enumerate(lens):
            new = 1 if case["form"] == "token" else n
            pos = torch.arange(n - new, n, device="cuda")
            turn = torch.polar(torch.ones(new, d // 2, dtype=torch.float64, device="cuda"),
                               pos.double()[:, None] * case["pi"] * theta)[:, None]
            for x in (q_rot, k_rot):
                y = torch.complex(x[row:row + new, :, :d // 2], x[row:row + new, :, d // 2:]) * turn
                x[row:row + new] = torch.cat((y.real, y.imag), -1)
            pages = torch.tensor(table[b], device="cuda")[pos // case["page"]].long()
            kc[pages, pos % case["page"]] = k_rot[row:row + new]
            vc[pages, pos % case["page"]] = s["v"][row:row + new].double()
            row += new
        return dict(q_rot=q_rot, k_rot=k_rot, k_cache=kc, v_cache=vc)
    if case["op"] == "decode":
        table = s["table"].tolist()
        o = torch.zeros(len(lens), hq, d, dtype=torch.float64, device="cuda")
        lse = torch.full((len(lens), hq), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            if n:
                at = torch.tensor([p for p in table[b] if p >= 0], device="cuda")
                k, v = (x[at].flatten(0, 1)[:n] for x in (s["k_cache"], s["v_cache"]))
                for h in range(hkv):
                    x, y = _attend64(s["q"][b, h * g:(h + 1) * g, None].double(), k[:, h].double(),
                                     v[:, h].double(), s["scale"], n - 1)
                    o[b, h * g:(h + 1) * g], lse[b, h * g:(h + 1) * g] = x[:, 0], y[:, 0]
        return dict(o=o, lse=lse)
    t = sum(lens)
    o = torch.empty(t, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(hq, t, dtype=torch.float64, device="cuda")
    rows, row = 2048, 0
    for n in lens:
        for h in range(hkv):
            q = s["q"][row:row + n, h * g:(h + 1) * g].double().permute(1, 0, 2)
            k, v = s["k"][row:row + n, h].double(), s["v"][row:row + n, h].double()
            for i in range(0, n, rows):
                e = min(n, i + rows)
                x, y = _attend64(q[:, i:e], k[:e], v[:e], s["scale"], i)
                o[row + i:row + e, h * g:(h + 1) * g] = x.permute(1, 0, 2)
                lse[h * g:(h + 1) * g, row + i:row + e] = y
        row += n
    return dict(o=o, lse=lse)
