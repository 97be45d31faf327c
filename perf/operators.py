"""Measured cases of the operators around the paged decode: attention over a
prefix that a batch shares, the attention weight each cached key received, and
the eviction of the keys that received least.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits), or through the library where ``own`` is set.  ``exact`` is the same
result in 64 bits, sequence by sequence from the definitions:

* shared prefix: out, lse of the paged attention forward.  Sequences of one
  group hold the same pages first, ``prefix`` keys of them.
* key weights:   w_out[b, hk, j] = beta w[b, hk, j]
                 + sum over the rows i and heads h of group hk of
                   exp(s_ij - lse[h, i])  over the visible (i, j).
* eviction:      a sequence of more than ``budget`` keys keeps its first
                 ``sink``, its last ``recent`` and, of the others, those of
                 largest weight (ties: the lowest index), in their order, moved
                 to the pages of a second table.

The sizes follow the library's paged decode benchmark (64 sequences of 512 to
8192 keys, 32 query heads over 8 kv heads of dim 128, pages of 16), its paged
e4m3 prefill (Q/K 192, V 128, pages of 64, 16 heads, lengths 1 to 4096), its
packed prefill (16 heads, 8 lengths up to 2048) and its small dense one (heads
of dim 64); the others are generic.
"""
import math
import random

import torch

own = False

_DEV = "cuda"


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a few chats behind one system prompt, one token each: latency
        dict(name="prefix_4seq_512_bf16", op="prefix", groups=1, seqs=4, plen_lo=512, plen_hi=512, slen_lo=1,
             slen_hi=64, sq=1, hq=32, hkv=8, d=128, page=16, kv="bf16", causal=True, window=0, mod="none",
             lens_seed=1),
        # a full decode batch behind one long instruction
        dict(name="prefix_64seq_8192_bf16", op="prefix", groups=1, seqs=64, plen_lo=8192, plen_hi=8192, slen_lo=16,
             slen_hi=1024, sq=1, hq=32, hkv=8, d=128, page=16, kv="bf16", causal=False, window=0, mod="none",
             lens_seed=2),
        # several prompts in one batch, drafts of up to 3 tokens to verify, byte cache, soft-cap
        dict(name="prefix_5groups_77seq_e4m3", op="prefix", groups=5, seqs=77, plen_lo=640, plen_hi=6000,
             slen_lo=3, slen_hi=700, sq=3, hq=16, hkv=4, d=128, page=64, kv="e4m3", causal=True, window=0,
             mod="softcap", lens_seed=3),
        # a document that many users ask about
        dict(name="prefix_192seq_65536_int8", op="prefix", groups=1, seqs=192, plen_lo=65536, plen_hi=65536,
             slen_lo=1, slen_hi=2048, sq=1, hq=32, hkv=8, d=128, page=64, kv="int8", causal=False, window=0,
             mod="none", lens_seed=4),
        # small heads, one kv head a query head, pages of few keys
        dict(name="prefix_17seq_1500_d64_bf16", op="prefix", groups=2, seqs=17, plen_lo=1000, plen_hi=1500,
             slen_lo=2, slen_hi=300, sq=2, hq=12, hkv=12, d=64, page=8, kv="bf16", causal=True, window=0,
             mod="alibi", lens_seed=5),
        # one token of each running sequence, after every decode step
        dict(name="weights_decode_64seq_bf16", op="weights", seqs=64, klen_lo=512, klen_hi=8192, sq=1, hq=32, hkv=8,
             d=128, page=16, kv="bf16", causal=True, window=0, mod="none", beta=1.0, lens_seed=6),
        # a small batch with a draft of 2, byte cache, decaying weights: latency
        dict(name="weights_decode_3seq_e4m3", op="weights", seqs=3, klen_lo=100, klen_hi=2500, sq=2, hq=16, hkv=4,
             d=128, page=64, kv="e4m3", causal=True, window=0, mod="softcap", beta=0.75, lens_seed=7),
        # the prompts themselves: every query row of a packed prefill
        dict(name="weights_prefill_8seq_bf16", op="weights", seqs=8, klen_lo=0, klen_hi=2048, sq=0, hq=16, hkv=16,
             d=128, page=0, kv="bf16", causal=True, window=0, mod="none", beta=0.0, lens_seed=8),
        # long prompts over a byte cache with Q/K heads of 192
        dict(name="weights_prefill_16seq_d192_e4m3", op="weights", seqs=16, klen_lo=1, klen_hi=4096, sq=0, hq=16,
             hkv=4, d=192, page=64, kv="e4m3", causal=True, window=0, mod="none", beta=0.0, lens_seed=9),
        # one small sequence that has just outgrown its budget: latency
        dict(name="evict_2seq_1100_to_1024_bf16", op="evict", seqs=2, klen_lo=1050, klen_hi=1100, budget=1024, sink=4,
             recent=256, hkv=8, dk=128, dv=128, page=16, kv="bf16", lens_seed=10),
        # a decode batch cut to a quarter
        dict(name="evict_48seq_8192_to_2048_bf16", op="evict", seqs=48, klen_lo=512, klen_hi=8192, budget=2048,
             sink=16, recent=512, hkv=8, dk=128, dv=128, page=16, kv="bf16", lens_seed=11),
        # a few very long contexts in a byte cache, Q/K 192 and V 128
        dict(name="evict_3seq_100000_to_9000_e4m3", op="evict", seqs=3, klen_lo=60000, klen_hi=100000, budget=9000,
             sink=64, recent=1000, hkv=4, dk=192, dv=128, page=64, kv="e4m3", lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prefix", "weights", "weights", "evict"])
    kv = rng.choice(["bf16", "e4m3", "int8"])
    seed = rng.randrange(1 << 30)
    mod = rng.choice(["none", "none", "softcap", "alibi"])
    if op == "prefix":
        hkv = rng.choice([1, 2, 4, 8, 12])
        group = rng.choice([1, 2, 3, 4, 7, 8, 16])
        sq = rng.randint(1, max(1, min(4, 16 // group)))
        seqs = _log_int(rng, 1, 192)
        phi = _log_int(rng, 64, 65536)
        while seqs * phi * group * hkv > 192 * 65536 * 32:
            phi = max(64, phi // 2)
        return dict(op=op, groups=rng.randint(1, min(6, seqs)), seqs=seqs, plen_lo=rng.randint(1, phi), plen_hi=phi,
                    slen_lo=1, slen_hi=_log_int(rng, 4, 2048), sq=sq, hq=hkv * group, hkv=hkv,
                    d=rng.choice([64, 128]), page=rng.choice([1, 4, 8, 16, 32, 64, 128]), kv=kv,
                    causal=rng.random() < 0.6, window=rng.choice([0, 0, 0, rng.randint(1, phi)]), mod=mod,
                    lens_seed=seed)
    if op == "weights":
        hkv = rng.choice([1, 2, 4, 8, 16])
        group = rng.choice([1, 2, 3, 4, 8])
        c = dict(op=op, hq=hkv * group, hkv=hkv, kv=kv, causal=rng.random() < 0.7,
                 window=rng.choice([0, 0, 0, rng.randint(1, 2000)]), mod=mod, beta=rng.choice([0.0, 0.5, 1.0]),
                 page=rng.choice([0, 1, 8, 16, 64, 256]), lens_seed=seed)
        if rng.random() < 0.5:   # decode and drafts
            c.update(seqs=_log_int(rng, 1, 64), klen_lo=rng.randint(0, 200), klen_hi=_log_int(rng, 201, 8192),
                     sq=rng.randint(1, 5), d=rng.choice([64, 128, 192]))
        else:                    # prompts
            c.update(seqs=_log_int(rng, 1, 16), klen_lo=rng.randint(0, 60), klen_hi=_log_int(rng, 61, 2900), sq=0,
                     d=rng.choice([64, 128, 192]))
        return c
    budget = _log_int(rng, 16, 9000)
    sink = rng.randint(0, min(64, budget // 4))
    dk, dv = rng.choice([(64, 64), (128, 128), (192, 128)])
    hi = _log_int(rng, budget // 2 + 1, 100000)
    seqs = _log_int(rng, 1, 48)
    while seqs * hi > 48 * 8192:
        seqs = max(1, seqs // 2)
        if seqs == 1:
            break
    return dict(op=op, seqs=seqs, klen_lo=rng.randint(0, hi), klen_hi=hi, budget=budget, sink=sink,
                recent=rng.randint(0, budget - sink), hkv=rng.choice([1, 2, 4, 8]), dk=dk, dv=dv,
                page=rng.choice([1, 4, 16, 64, 256]), kv=kv, lens_seed=seed)


# ----------------------------------------------------------------- lengths --

def _geometry(case):
    """Lengths of a case, from the case alone."""
    rng = random.Random(case["lens_seed"])
    n = case["seqs"]
    g = {}
    if case["op"] == "prefix":
        page = case["page"]
        cuts = sorted(rng.randint(0, n) for _ in range(case["groups"] - 1))
        g["cu_groups"] = [0] + cuts + [n]
        # whole pages are shared
        g["prefix"] = [rng.randint(case["plen_lo"], case["plen_hi"]) // page * page for _ in range(case["groups"])]
        g["group_of"] = []
        for x in range(case["groups"]):
            g["group_of"] += [x] * (g["cu_groups"][x + 1] - g["cu_groups"][x])
        # now and then a slot of the batch that has nothing to ask
        g["q_lens"] = [case["sq"] if rng.random() < 0.9 else rng.randint(0, case["sq"]) for _ in range(n)]
        g["q_lens"][rng.randrange(n)] = case["sq"]
        g["k_lens"] = [g["prefix"][g["group_of"][b]] + max(rng.randint(case["slen_lo"], case["slen_hi"]), g["q_lens"][b])
                       for b in range(n)]
        return g
    g["k_lens"] = [rng.randint(case["klen_lo"], case["klen_hi"]) for _ in range(n)]
    g["k_lens"][rng.randrange(n)] = case["klen_hi"]
    if case["op"] == "weights":
        if case["sq"]:
            g["q_lens"] = [min(case["sq"], x) if case["causal"] else case["sq"] for x in g["k_lens"]]
        else:
            # whole prompts, and now and then the last piece of one
            g["q_lens"] = [x if rng.random() < 0.75 else rng.randint(0, x) for x in g["k_lens"]]
        if sum(g["q_lens"]) == 0:
            g["q_lens"][0] = 1
            g["k_lens"][0] = max(1, g["k_lens"][0])
    return g


def _visible(case, g):
    """Visible (row, key) pairs of all sequences, one head."""
    total = 0
    for nq, nk in zip(g["q_lens"], g["k_lens"]):
        for i in range(nq):
            p = i + nk - nq
            lo, hi = 0, nk
            if case["causal"]:
                hi = min(hi, p + 1)
            if case["window"] > 0:
                lo = max(lo, p - case["window"] + 1)
                if not case["causal"]:
                    hi = min(hi, p + case["window"])
            total += max(0, hi - lo)
    return total


def _esz(kv):
    return 2 if kv == "bf16" else 1


def work(case):
    g = _geometry(case)
    esz, hkv = _esz(case["kv"]), case["hkv"]
    scale = 0 if case["kv"] == "bf16" else 4
    if case["op"] == "evict":
        moved = sum(min(x, case["budget"]) for x in g["k_lens"])
        row = (case["dk"] + case["dv"]) * esz + 2 * scale
        # weights in, rows in and out, weights and kept indices out
        return {"bytes": 4 * hkv * sum(g["k_lens"]) + hkv * moved * (2 * row + 8), "flops": 0}
    tq, d, hq = sum(g["q_lens"]), case["d"], case["hq"]
    pairs = _visible(case, g)
    if case["op"] == "prefix":
        shared = [p for p, lo, hi in zip(g["prefix"], g["cu_groups"], g["cu_groups"][1:]) if hi > lo]
        own_keys = sum(k - g["prefix"][x] for k, x in zip(g["k_lens"], g["group_of"]))
        keys = sum(shared) + own_keys
        return {"bytes": keys * hkv * 2 * (d * esz + scale) + tq * hq * (4 * d + 4), "flops": 4 * d * hq * pairs}
    keys = sum(k for k, q in zip(g["k_lens"], g["q_lens"]) if q)
    io = 4 * hkv * sum(g["k_lens"]) * (2 if case["beta"] else 1)
    return {"bytes": keys * hkv * (d * esz + scale) + io + tq * hq * (2 * d + 4), "flops": 2 * d * hq * pairs}


# ------------------------------------------------------------------ inputs --

def _quantize(x, kv):
    """(stored values, per-token scales or None) of fp32 [..., D]."""
    if kv == "bf16":
        return x.to(torch.bfloat16), None
    top = 448.0 if kv == "e4m3" else 127.0
    scale = x.abs().amax(-1) / top
    y = x / torch.where(scale > 0, scale, torch.ones_like(scale)).unsqueeze(-1)
    y = y.to(torch.float8_e4m3fn) if kv == "e4m3" else y.round().clamp_(-127, 127).to(torch.int8)
    return y, scale


def _cu(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(_DEV)


def _pages(lens, page, gen, first=0, spare=3):
    """Shuffled pages for sequences of these lengths: table [B, max] (-1 past a sequence's end), pages in all."""
    need = [(x + page - 1) // page for x in lens]
    ids = torch.randperm(sum(need) + spare, generator=gen, device=_DEV).to(torch.int32) + first
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device=_DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, sum(need) + spare


def _keys(rows, hkv, d, gen, heavy):
    """Keys with a shared direction that a few of them (the sinks, some words) carry strongly."""
    k = torch.randn((rows, hkv, d), generator=gen, device=_DEV)
    if heavy is not None:
        hit = (torch.rand((rows, hkv, 1), generator=gen, device=_DEV) < 0.01).float()
        k += 2.5 * hit * heavy
    return k


def _mod_args(case):
    if case["mod"] == "softcap":
        return dict(softcap=20.0)
    if case["mod"] == "alibi":
        return dict(alibi_slope=0.01)
    return {}


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed)
    g = _geometry(case)
    hkv, kv, page = case["hkv"], case["kv"], case["page"]
    st = dict(case=case, geo=g)
    if case["op"] == "evict":
        lens = g["k_lens"]
        st["bt"], n1 = _pages(lens, page, gen)
        st["bt_out"], n2 = _pages([min(x, case["budget"]) for x in lens], page, gen, first=n1)
        for name, d in (("k", case["dk"]), ("v", case["dv"])):
            x, s = _quantize(_keys((n1 + n2) * page, hkv, d, gen, None), kv)
            st[name] = x.view(n1 + n2, page, hkv, d)
            st[name + "_scale"] = None if s is None else s.view(n1 + n2, page, hkv)
        # accumulated weights: most keys get little, a few much, some the very same
        w = torch.exp(2.0 * torch.randn((case["seqs"], hkv, max(1, max(lens))), generator=gen, device=_DEV) - 3.0)
        st["w"] = torch.where(w < 0.02, torch.floor(w * 256) / 256, w)
        st["w_out"] = torch.empty((case["seqs"], hkv, case["budget"]), device=_DEV)
        st["cu_k"] = _cu(lens)
        return st
    d, hq = case["d"], case["hq"]
    heavy = torch.randn((1, hkv, d), generator=gen, device=_DEV)
    heavy /= heavy.norm(dim=-1, keepdim=True)
    tq = sum(g["q_lens"])
    q = torch.randn((tq, hq, d), generator=gen, device=_DEV) + 2.0 * heavy.repeat_interleave(hq // hkv, 1)
    st["q"] = q.to(torch.bfloat16)
    st["cu_q"], st["cu_k"] = _cu(g["q_lens"]), _cu(g["k_lens"])
    if case["op"] == "prefix":
        # a group's pages first, then each sequence's own
        pre, n1 = _pages(g["prefix"], page, gen)
        own_lens = [k - g["prefix"][x] for k, x in zip(g["k_lens"], g["group_of"])]
        suf, n2 = _pages(own_lens, page, gen, first=n1)
        width = max(1, max((k + page - 1) // page for k in g["k_lens"]))
        st["bt"] = torch.full((case["seqs"], width), -1, dtype=torch.int32, device=_DEV)
        for b, x in enumerate(g["group_of"]):
            np_, ns = g["prefix"][x] // page, (own_lens[b] + page - 1) // page
            st["bt"][b, :np_] = pre[x, :np_]
            st["bt"][b, np_:np_ + ns] = suf[b, :ns]
        shape = (n1 + n2, page)
        st["cu_groups"] = torch.tensor(g["cu_groups"], dtype=torch.int32, device=_DEV)
        st["prefix_lens"] = torch.tensor(g["prefix"], dtype=torch.int32, device=_DEV)
    elif page:
        st["bt"], n = _pages(g["k_lens"], page, gen)
        shape = (n, page)
    else:
        st["bt"] = None
        shape = (max(1, sum(g["k_lens"])),)
    rows = math.prod(shape)
    x, s = _quantize(_keys(rows, hkv, d, gen, heavy), kv)
    st["k"] = x.view(*shape, hkv, d)
    st["k_scale"] = None if s is None else s.view(*shape, hkv)
    if case["op"] == "prefix":
        x, s = _quantize(_keys(rows, hkv, d, gen, None), kv)
        st["v"] = x.view(*shape, hkv, d)
        st["v_scale"] = None if s is None else s.view(*shape, hkv)
        if own:
            st["plan"] = _prefix_plan(st)
        return st
    width = max(1, max(g["k_lens"]))
    st["w"] = torch.rand((case["seqs"], hkv, width), generator=gen, device=_DEV) if case["beta"] else None
    st["w_out"] = torch.empty((case["seqs"], hkv, width), device=_DEV)
    # the forward's lse of the same call
    st["lse"] = torch.empty((hq, tq), device=_DEV)
    for bs, s_, ok in _padded_scores(st):
        s_ = torch.where(ok, s_, -math.inf).logsumexp(-1)   # [b, hkv, group, Lq]
        for x, b in enumerate(bs):
            n, at = g["q_lens"][b], sum(g["q_lens"][:b])
            st["lse"][:, at:at + n] = s_[x, :, :, :n].reshape(hq, n)
    if own and case["sq"]:
        st["plan"] = _weights_plan(st)
    return st


# -------------------------------------------------------------- plain forms --

def _rows_of(st, b, lo, hi):
    """Rows of the flat [tokens, Hkv, D] cache that hold keys lo .. hi-1 of sequence b."""
    j = torch.arange(lo, hi, device=_DEV)
    if st["bt"] is None:
        return j + sum(st["geo"]["k_lens"][:b])
    page = st["case"]["page"]
    return st["bt"][b].long()[j // page] * page + j % page


def _as_stored(x):
    """The cache as flat [tokens, Hkv, D] rows: bf16 values, or the bytes of the others."""
    x = x.reshape(-1, *x.shape[-2:])
    return x if x.dtype == torch.bfloat16 else x.view(torch.uint8)


def _values(st, name, rows):
    """fp32 [len(rows), Hkv, D] that the stored keys or values stand for."""
    x = _as_stored(st[name])[rows].view(st[name].dtype).float()
    s = st[name + "_scale"]
    return x if s is None else x * s.reshape(-1, s.shape[-1])[rows].unsqueeze(-1)


def _modified(case, s, dist):
    """Soft-cap or ALiBi on scaled scores; dist = i' - j."""
    if case["mod"] == "softcap":
        return 20.0 * torch.tanh(s / 20.0)
    if case["mod"] == "alibi":
        return s - 0.01 * dist.abs()
    return s


def _allowed(case, dist):
    ok = torch.ones_like(dist, dtype=torch.bool)
    if case["causal"]:
        ok &= dist >= 0
    if case["window"] > 0:
        ok &= (dist < case["window"]) & (dist > -case["window"])
    return ok


def _padded_scores(st):
    """Scores of a few sequences at a time, padded to their longest: yields
    (sequences, scores [b, Hkv, group, Lq, Lk], visible)."""
    case, g = st["case"], st["geo"]
    hkv, d = case["hkv"], case["d"]
    group = case["hq"] // hkv
    order = [b for b in range(case["seqs"]) if g["q_lens"][b]]
    at = 0
    while at < len(order):
        bs, lq, lk = [], 0, 1
        while at < len(order):
            q2, k2 = max(lq, g["q_lens"][order[at]]), max(lk, g["k_lens"][order[at]])
            if bs and (len(bs) + 1) * k2 * max(case["hq"] * q2, hkv * d) > 1 << 28:
                break
            bs.append(order[at])
            lq, lk = q2, k2
            at += 1
        q = torch.zeros((len(bs), lq, hkv, group, d), device=_DEV)
        k = torch.zeros((len(bs), lk, hkv, d), device=_DEV)
        dist = torch.zeros((len(bs), lq, lk), dtype=torch.int64, device=_DEV)
        real = torch.zeros((len(bs), lq, lk), dtype=torch.bool, device=_DEV)
        i, j = torch.arange(lq, device=_DEV), torch.arange(lk, device=_DEV)
        for x, b in enumerate(bs):
            nq, nk, q0 = g["q_lens"][b], g["k_lens"][b], sum(g["q_lens"][:b])
            q[x, :nq] = st["q"][q0:q0 + nq].float().view(nq, hkv, group, d)
            k[x, :nk] = _values(st, "k", _rows_of(st, b, 0, nk))
            dist[x] = (i[:, None] + nk - nq) - j[None, :]
            real[x, :nq, :nk] = True
        s = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(len(bs), hkv, group * lq, d), k.permute(0, 2, 3, 1))
        s = s.view(len(bs), hkv, group, lq, lk) / math.sqrt(d)
        dist = dist[:, None, None]
        yield bs, _modified(case, s, dist), _allowed(case, dist) & real[:, None, None]


def _plain_prefix(st):
    case, g = st["case"], st["geo"]
    hkv, d, hq = case["hkv"], case["d"], case["hq"]
    group = hq // hkv
    tq = sum(g["q_lens"])
    out = torch.zeros((tq, hq, d), dtype=torch.bfloat16, device=_DEV)
    lse = torch.full((hq, tq), -math.inf, device=_DEV)
    for x in range(case["groups"]):
        seqs = [b for b in range(g["cu_groups"][x], g["cu_groups"][x + 1]) if g["q_lens"][b]]
        if not seqs:
            continue
        n = sum(g["q_lens"][b] for b in seqs)
        q0 = sum(g["q_lens"][:seqs[0]])
        plen = g["prefix"][x]
        ls = max(g["k_lens"][b] - plen for b in seqs)
        pos = torch.cat([torch.arange(g["q_lens"][b], device=_DEV) + g["k_lens"][b] - g["q_lens"][b] for b in seqs])
        end = torch.cat([torch.full((g["q_lens"][b],), g["k_lens"][b], device=_DEV) for b in seqs])
        q = st["q"][q0:q0 + n].float().view(n, hkv, group, d) / math.sqrt(d)
        # the shared keys once for all rows of the group
        rows = _rows_of(st, seqs[0], 0, plen)
        kp, vp = _values(st, "k", rows), _values(st, "v", rows)
        qh = q.permute(1, 0, 2, 3).reshape(hkv, n * group, d)
        s = torch.empty((hkv, n, group, plen + ls), device=_DEV)
        s[..., :plen] = torch.matmul(qh, kp.permute(1, 2, 0)).view(hkv, n, group, plen)
        # each sequence's own
        at, vs = 0, []
        for b in seqs:
            m, own_keys = g["q_lens"][b], g["k_lens"][b] - plen
            rows = _rows_of(st, b, plen, g["k_lens"][b])
            ks = _values(st, "k", rows)
            vs.append(_values(st, "v", rows))
            s[:, at:at + m, :, plen:plen + own_keys] = torch.matmul(
                q[at:at + m].permute(1, 0, 2, 3).reshape(hkv, m * group, d),
                ks.permute(1, 2, 0)).view(hkv, m, group, own_keys)
            at += m
        j = torch.arange(plen + ls, device=_DEV)
        dist = (pos[:, None] - j[None, :])[None, :, None, :]
        ok = _allowed(case, dist) & (j[None, :] < end[:, None])[None, :, None, :]
        s = torch.where(ok, _modified(case, s, dist), -math.inf)
        top = s.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        p = torch.exp(s - top)
        den = p.sum(-1, keepdim=True)
        o = torch.matmul(p[..., :plen].reshape(hkv, n * group, plen), vp.permute(1, 0, 2)).view(hkv, n, group, d)
        at = 0
        for b, v in zip(seqs, vs):
            m = g["q_lens"][b]
            o[:, at:at + m] += torch.matmul(p[:, at:at + m, :, plen:plen + v.shape[0]].reshape(hkv, m * group, -1),
                                            v.permute(1, 0, 2)).view(hkv, m, group, d)
            at += m
        o = torch.where(den > 0, o / den, torch.zeros_like(o))
        out[q0:q0 + n] = o.permute(1, 0, 2, 3).reshape(n, hq, d).to(torch.bfloat16)
        lse[:, q0:q0 + n] = (top + torch.log(den))[..., 0].permute(0, 2, 1).reshape(hq, n)
    return out, lse


def _plain_weights(st):
    case, g = st["case"], st["geo"]
    hkv = case["hkv"]
    group = case["hq"] // hkv
    w = st["w"] * case["beta"] if st["w"] is not None else torch.zeros_like(st["w_out"])
    for bs, s, ok in _padded_scores(st):
        for x, b in enumerate(bs):
            nq, nk, q0 = g["q_lens"][b], g["k_lens"][b], sum(g["q_lens"][:b])
            lse = st["lse"][:, q0:q0 + nq].view(hkv, group, nq, 1)
            seen = ok[x, :, :, :nq, :nk]
            p = torch.exp(torch.where(seen, s[x, :, :, :nq, :nk] - lse, -math.inf))
            w[b, :, :nk] += p.sum((1, 2))
    return w


def _plain_evict(st):
    case = st["case"]
    w, budget, hkv, page = st["w"], case["budget"], case["hkv"], case["page"]
    n, _, width = w.shape
    lens = (st["cu_k"][1:] - st["cu_k"][:-1]).long()
    keep = lens.clamp(max=budget)
    j = torch.arange(width, device=_DEV)
    real = (j[None, :] < lens[:, None])[:, None]
    held = (j < case["sink"])[None, None] | (j[None, :] >= (lens - case["recent"])[:, None])[:, None]
    held = held | (lens <= budget)[:, None, None]
    rank = torch.where(real, torch.where(held, math.inf, w), -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    if width < budget:
        order = torch.nn.functional.pad(order, (0, budget - width))
    slot = torch.arange(budget, device=_DEV)
    live = (slot[None, :] < keep[:, None])[:, None].expand(n, hkv, budget)
    kept = torch.where(live, order[..., :budget], width).sort(-1).values
    b, h, r = torch.nonzero(live, as_tuple=True)
    src_j = kept[b, h, r]
    src = st["bt"][b, src_j // page].long() * page + src_j % page
    dst = st["bt_out"][b, r // page].long() * page + r % page
    for name in ("k", "v"):
        raw = _as_stored(st[name])
        raw[dst, h] = raw[src, h]
        s = st[name + "_scale"]
        if s is not None:
            s = s.view(-1, hkv)
            s[dst, h] = s[src, h]
    st["w_out"].zero_()
    st["w_out"][b, h, r] = w[b, h, src_j]
    kept = torch.where(live, kept, -1).to(torch.int32)
    cu = torch.cat([torch.zeros_like(keep[:1]), keep.cumsum(0)]).to(torch.int32)
    return _evicted(st, kept, cu)


def _evicted(st, kept, cu):
    out = dict(kept=kept, cu_seqlens_k=cu, weights=st["w_out"])
    for name in ("k", "v"):
        x = st[name]
        out[name] = x if x.dtype == torch.bfloat16 else x.view(torch.uint8)   # moved as stored
        if st[name + "_scale"] is not None:
            out[name + "_scale"] = st[name + "_scale"]
    return out


# --------------------------------------------------------- the library's calls --

def _lib():
    import flashattention_forward_gb300 as fa
    return fa


def _attention_args(st):
    fa, case, g = _lib(), st["case"], st["geo"]
    kind = dict(none=fa.MOD_NONE, softcap=fa.MOD_SOFTCAP, alibi=fa.MOD_ALIBI)[case["mod"]]
    return dict(max_seqlen_q=max(g["q_lens"]), max_seqlen_k=max(g["k_lens"]), block_table=st["bt"],
                page_size=case["page"], k_scale=st["k_scale"], causal=case["causal"], window=case["window"],
                score_mod=kind, **_mod_args(case))


def _prefix_plan(st):
    """A decode loop prepares the call once and repeats it."""
    g = st["geo"]
    return _lib().SharedPrefixPlan(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], v_scale=st["v_scale"],
                                   cu_groups=st["cu_groups"], prefix_lens=st["prefix_lens"],
                                   max_prefix_len=max(g["prefix"]), total_k=sum(g["k_lens"]), **_attention_args(st))


def _weights_plan(st):
    return _lib().KeyWeightsPlan(st["q"], st["k"], st["lse"], st["cu_q"], st["cu_k"], weights=st["w"],
                                 beta=st["case"]["beta"], out=st["w_out"], **_attention_args(st))


def run(state):
    case = state["case"]
    if not own:
        return {"prefix": _plain_prefix, "weights": _plain_weights, "evict": _plain_evict}[case["op"]](state)
    fa = _lib()
    if "plan" in state:
        return state["plan"].run()
    if case["op"] == "weights":
        return fa.key_weights(state["q"], state["k"], state["lse"], state["cu_q"], state["cu_k"],
                              weights=state["w"], beta=case["beta"], out=state["w_out"], **_attention_args(state))
    kept, cu = fa.cache_evict(state["w"], state["k"], state["v"], state["cu_k"], block_table=state["bt"],
                              page_size=case["page"], budget=case["budget"], sink=case["sink"],
                              recent=case["recent"], max_seqlen_k=max(state["geo"]["k_lens"]),
                              k_scale=state["k_scale"], v_scale=state["v_scale"], block_table_out=state["bt_out"],
                              weights_out=state["w_out"])
    return _evicted(state, kept, cu)


# --------------------------------------------------------------- 64 bits --

def exact(case, seed):
    st = prepare(case, seed)
    g = st["geo"]
    f64 = torch.float64

    def stored(name, rows, h):
        x = _as_stored(st[name])[rows, h].view(st[name].dtype).to(f64)
        s = st[name + "_scale"]
        return x if s is None else x * s.reshape(-1, s.shape[-1])[rows, h].to(f64)[:, None]

    def cache_rows(b):
        n = g["k_lens"][b]
        if st["bt"] is None:
            start = sum(g["k_lens"][:b])
            return torch.arange(start, start + n, device=_DEV)
        table = st["bt"][b].tolist()
        pg = case["page"]
        pages = torch.tensor([table[x] for x in range((n + pg - 1) // pg)], dtype=torch.int64, device=_DEV)
        return (pages[:, None] * pg + torch.arange(pg, device=_DEV)[None]).reshape(-1)[:n]

    if case["op"] == "evict":
        budget, sink, recent = case["budget"], case["sink"], case["recent"]
        w = st["w"].cpu().tolist()
        kept = torch.full((case["seqs"], case["hkv"], budget), -1, dtype=torch.int32)
        wout = torch.zeros((case["seqs"], case["hkv"], budget), dtype=f64)
        total, cu = 0, [0]
        for b, n in enumerate(g["k_lens"]):
            m = min(n, budget)
            total += m
            cu.append(total)
            rows = cache_rows(b) if n else None
            pg = case["page"]
            to = st["bt_out"][b].tolist()
            dst = torch.tensor([to[r // pg] * pg + r % pg for r in range(m)], dtype=torch.int64, device=_DEV)
            for h in range(case["hkv"]):
                if n <= budget:
                    pick = list(range(n))
                else:
                    mid = sorted(range(sink, n - recent), key=lambda x: (-w[b][h][x], x))[:budget - sink - recent]
                    pick = list(range(sink)) + sorted(mid) + list(range(n - recent, n))
                if not pick:
                    continue
                kept[b, h, :m] = torch.tensor(pick, dtype=torch.int32)
                wout[b, h, :m] = torch.tensor([w[b][h][x] for x in pick], dtype=f64)
                src = rows[torch.tensor(pick, dtype=torch.int64, device=_DEV)]
                for name in ("k", "v"):
                    raw = _as_stored(st[name])
                    raw[dst, h] = raw[src, h]
                    if st[name + "_scale"] is not None:
                        s = st[name + "_scale"].view(-1, case["hkv"])
                        s[dst, h] = s[src, h]
        res = _evicted(st, kept.to(_DEV), torch.tensor(cu, dtype=torch.int32, device=_DEV))
        res["weights"] = wout.to(_DEV)
        return res

    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    group = hq // hkv
    tq = sum(g["q_lens"])
    if case["op"] == "prefix":
        out = torch.zeros((tq, hq, d), dtype=f64, device=_DEV)
        lse = torch.full((hq, tq), -math.inf, dtype=f64, device=_DEV)
    else:
        w = torch.zeros(st["w_out"].shape, dtype=f64, device=_DEV)
        if st["w"] is not None:
            w += case["beta"] * st["w"].to(f64)
    q0 = 0
    for b, (nq, nk) in enumerate(zip(g["q_lens"], g["k_lens"])):
        if nq == 0 or nk == 0:
            q0 += nq
            continue
        rows = cache_rows(b)
        dist = torch.arange(nq, device=_DEV)[:, None] + (nk - nq) - torch.arange(nk, device=_DEV)[None]
        hidden = torch.zeros_like(dist, dtype=torch.bool)
        if case["causal"]:
            hidden |= dist < 0
        if case["window"] > 0:
            hidden |= dist >= case["window"]
            hidden |= dist <= -case["window"]
        for hk in range(hkv):
            k = stored("k", rows, hk)
            for h in range(hk * group, (hk + 1) * group):
                s = st["q"][q0:q0 + nq, h].to(f64) @ k.T * d ** -0.5
                if case["mod"] == "softcap":
                    s = 20.0 * torch.tanh(s / 20.0)
                elif case["mod"] == "alibi":
                    s = s - 0.01 * dist.abs()
                s.masked_fill_(hidden, -math.inf)
                if case["op"] == "prefix":
                    z = torch.logsumexp(s, -1)
                    lse[h, q0:q0 + nq] = z
                    p = torch.exp(s - z[:, None]).masked_fill_(hidden, 0.0)
                    out[q0:q0 + nq, h] = p @ stored("v", rows, hk)
                else:
                    z = st["lse"][h, q0:q0 + nq].to(f64)[:, None]
                    w[b, hk, :nk] += torch.exp(s - z).masked_fill_(hidden, 0.0).sum(0)
        q0 += nq
    return (out, lse) if case["op"] == "prefix" else w
