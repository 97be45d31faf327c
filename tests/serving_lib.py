"""Inputs and 64-bit references for the operators around the paged decode
(shared prefixes, key weights, eviction).  Sequence by sequence, from the
definitions; every slot of the cache that no key occupies holds NaN (bf16,
e4m3, scales) or the type's extreme (int8).

Tolerances, derived from the roundings a kernel may make:
 * a score is an fp32 sum of D exact products, then a few fp32 operations:
   off by at most eps_s = (D + 8) 2^-24 scale sum_d |q_d k_d| + 2^-21 |s|;
 * a weight exp(s - LSE) is off by a factor of about eps_s + 2^-20 (ex2 and the
   fp32 LSE), a sum of n of them by 2^-24 (n / 128 + 128) more;
 * out: each weight rounded to bf16 before P V (2^-8 relative at most, also
   after the V scale), one rounding of the result: 2^-8 (sum w |v| + |out|).
"""
import math

import numpy as np
import torch

PAD = 7


def quantize(x, kv):
    if kv == "bf16":
        return x.to(torch.bfloat16), None
    top = 448.0 if kv == "e4m3" else 127.0
    s = (x.abs().amax(-1) / top).float()
    y = x / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(-1)
    return (y.to(torch.float8_e4m3fn) if kv == "e4m3" else y.round().clamp(-127, 127).to(torch.int8)), s


def poison(shape, kv):
    if kv == "bf16":
        return torch.full(shape, math.nan, dtype=torch.bfloat16), None
    if kv == "e4m3":
        x = torch.full(shape, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn)
    else:
        x = torch.full(shape, -128, dtype=torch.int8)
    return x, torch.full(shape[:-1], math.nan)


def raw(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


class Cache:
    """A paged (page > 0) or packed cache.  ``rows[b]``: row of the flat
    [tokens, Hkv, D] view of each key of sequence b."""

    def __init__(self, lens, hkv, dk, dv, page, kv, seed, prefix=None, groups=None, spare=3, extra_pages=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.kv, self.hkv = list(lens), page, kv, hkv
        self.dk, self.dv = dk, dv
        n = len(lens)
        if page:
            need = [(x + page - 1) // page for x in lens]
            shared = [0] * n
            if prefix is not None:
                for x in range(len(prefix)):
                    for b in range(groups[x], groups[x + 1]):
                        shared[b] = prefix[x] // page
            own = [max(0, a - s) for a, s in zip(need, shared)]
            total = sum(own) + sum(p // page for p in (prefix or [])) + spare + extra_pages
            ids = torch.randperm(total, generator=g).tolist()
            width = max(1, max(need + [p // page for p in (prefix or [0])]))
            bt = torch.full((n, width), -1, dtype=torch.int32)
            at = 0
            if prefix is not None:
                for x in range(len(prefix)):
                    k = prefix[x] // page
                    for b in range(groups[x], groups[x + 1]):
                        bt[b, :k] = torch.tensor(ids[at:at + k], dtype=torch.int32)
                    at += k
            for b in range(n):
                bt[b, shared[b]:shared[b] + own[b]] = torch.tensor(ids[at:at + own[b]], dtype=torch.int32)
                at += own[b]
            self.free = ids[at:]
            self.bt = bt
            shape = (total, page)
            self.rows = [torch.tensor([int(bt[b, j // page]) * page + j % page for j in range(lens[b])], dtype=torch.int64)
                         for b in range(n)]
        else:
            self.bt = None
            shape = (max(1, sum(lens)) + spare,)
            at = np.concatenate([[0], np.cumsum(lens)])
            self.rows = [torch.arange(int(at[b]), int(at[b + 1])) for b in range(n)]
        self.k, self.k_scale = poison((*shape, hkv, dk), kv)
        self.v, self.v_scale = poison((*shape, hkv, dv), kv)
        used = torch.unique(torch.cat(self.rows + [torch.zeros(0, dtype=torch.int64)]))
        if prefix is not None:   # whole pages are shared: every slot of them holds a key
            for x in range(len(prefix)):
                for b in range(groups[x], min(groups[x] + 1, groups[x + 1])):
                    j = torch.arange(prefix[x] // page * page)
                    used = torch.unique(torch.cat([used, self.bt[b][j // page].long() * page + j % page]))
        for name, d in (("k", dk), ("v", dv)):
            x, s = quantize(torch.randn((len(used), hkv, d), generator=g), kv)
            flat = raw(getattr(self, name)).view(-1, hkv, d)
            flat[used] = raw(x)
            if s is not None:
                getattr(self, name + "_scale").view(-1, hkv)[used] = s

    def values(self, name, rows):
        x = raw(getattr(self, name)).view(-1, self.hkv, getattr(self, "d" + name))[rows]
        x = x.view(getattr(self, name).dtype).double()
        s = getattr(self, name + "_scale")
        return x if s is None else x * s.view(-1, self.hkv)[rows].double().unsqueeze(-1)

    def to(self, dev):
        d = {n: getattr(self, n) for n in ("k", "v", "k_scale", "v_scale", "bt")}
        d = {n: None if t is None else t.to(dev) for n, t in d.items()}
        d["cu_k"] = cu(self.lens).to(dev)
        return d


def cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


def make_q(tq, hq, d, seed, strided=False):
    g = torch.Generator().manual_seed(seed + 1000)
    q = torch.randn((tq, hq, d), generator=g).to(torch.bfloat16)
    if strided:   # a view into a wider fused projection
        wide = torch.full((tq, hq + 2, d + 16), math.nan, dtype=torch.bfloat16)
        wide[:, 1:hq + 1, :d] = q
        q = wide[:, 1:hq + 1, :d]
    return q


def attention(q, q_lens, cache, k_lens, *, causal=False, window=0, mod="none", slope=0.0, cap=0.0, scale=None,
              want="out", lse=None, rows=None):
    """fp64 reference.  want "out": (out, lse, bound of out, bound of lse);
    want "weights": ([B, Hkv, max k] sums of exp(s - lse), bound)."""
    hq, d, hkv = q.shape[1], q.shape[2], cache.hkv
    grp = hq // hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    tq = sum(q_lens)
    rows = cache.rows if rows is None else rows
    out = torch.zeros((tq, hq, cache.dv), dtype=torch.float64)
    ref_lse = torch.full((hq, tq), -math.inf, dtype=torch.float64)
    b_out, b_lse = torch.zeros_like(out), torch.zeros_like(ref_lse)
    width = max([1] + list(k_lens))
    w = torch.zeros((len(q_lens), hkv, width), dtype=torch.float64)
    b_w = torch.zeros_like(w)
    at = 0
    for b, (nq, nk) in enumerate(zip(q_lens, k_lens)):
        if nq and nk:
            k = cache.values("k", rows[b][:nk])
            v = cache.values("v", rows[b][:nk]) if want == "out" else None
            dist = torch.arange(nq)[:, None] + nk - nq - torch.arange(nk)[None]
            ok = torch.ones((nq, nk), dtype=torch.bool)
            if causal:
                ok &= dist >= 0
            if window > 0:
                ok &= dist.abs() < window
                if causal:
                    ok &= dist < window
            for h in range(hq):
                qh, kh = q[at:at + nq, h].double(), k[:, h // grp]
                s = qh @ kh.T * scale
                eps = (d + 8) * 2.0 ** -24 * abs(scale) * (qh.abs() @ kh.abs().T) + 2.0 ** -21 * s.abs()
                if mod == "softcap":
                    s = cap * torch.tanh(s / cap)
                    eps = eps + 2.0 ** -20 * cap       # 1 / (1 + e^2u) near its ends
                elif mod == "alibi":
                    s = s - slope * dist.abs()
                    eps = eps + 2.0 ** -21 * slope * dist.abs()
                s = torch.where(ok, s, -math.inf)
                eps = torch.where(ok, eps, 0.0)
                z = torch.logsumexp(s, -1)
                if want == "out":
                    ref_lse[h, at:at + nq] = z
                    e = eps.amax(-1)
                    b_lse[h, at:at + nq] = e + 2.0 ** -20 * (1 + torch.where(z == -math.inf, 0.0, z).abs())
                    p = torch.where(ok, torch.exp(s - z[:, None]), 0.0)
                    vh = v[:, h // grp]
                    o = p @ vh
                    out[at:at + nq, h] = o
                    b_out[at:at + nq, h] = (2.0 ** -8 + 2 * e[:, None]) * (p @ vh.abs()) + 2.0 ** -8 * o.abs() + 1e-7
                else:
                    zz = (z if lse is None else lse[h, at:at + nq].double())[:, None]
                    p = torch.where(ok & (zz != -math.inf), torch.exp(s - zz), 0.0)
                    w[b, h // grp, :nk] += p.sum(0)
                    rel = eps + 2.0 ** -20 * (1 + torch.where(zz == -math.inf, 0.0, zz).abs()) + \
                        2.0 ** -24 * (nq * grp / 128 + 128)
                    b_w[b, h // grp, :nk] += (p * rel).sum(0) + 1e-30
        at += nq
    if want == "out":
        return out, ref_lse, b_out, b_lse
    return w, b_w


def within(got, ref, bound):
    """max |got - ref| / bound; infinite entries must be the same."""
    got = got.double().cpu()
    assert got.shape == ref.shape
    assert not torch.isnan(got).any()
    inf = torch.isinf(ref)
    assert torch.equal(torch.where(inf, got, torch.zeros_like(got)), torch.where(inf, ref, torch.zeros_like(ref)))
    x = torch.where(inf, torch.zeros_like(ref), (got - ref).abs() - bound)
    worst = float(x.max()) if x.numel() else 0.0
    assert worst <= 0, f"off by {worst} more than the bound"


def evict(weights, lens, budget, sink, recent):
    """(kept [B, Hkv, budget], new lengths) by a plain sort."""
    b, hkv, _ = weights.shape
    kept = torch.full((b, hkv, budget), -1, dtype=torch.int32)
    for x in range(b):
        n = lens[x]
        for h in range(hkv):
            if n <= budget:
                pick = list(range(n))
            else:
                w = weights[x, h].tolist()
                w = [(-math.inf, 0) if math.isnan(y) else (y, 1) for y in w]     # NaN below -inf
                mid = sorted(range(sink, n - recent), key=lambda j: (-w[j][0], -w[j][1], j))[:budget - sink - recent]
                pick = sorted(list(range(sink)) + mid + list(range(n - recent, n)))
            kept[x, h, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
    return kept, [min(n, budget) for n in lens]
