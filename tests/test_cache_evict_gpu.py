"""Eviction from a paged cache against a plain sort (serving_lib.evict): the
kept indices, moved rows, scales and weights are compared exactly."""
import math

import pytest
import torch

import serving_lib as sl

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from flashattention_forward_gb300 import build
    build.build()
    yield
    import flashattention_forward_gb300 as fa
    assert fa.device_error() == 0


def bits(x):
    return None if x is None else x.contiguous().view(torch.uint8).cpu()


def run(lens, budget, sink=0, recent=0, hkv=2, dk=128, dv=128, page=16, kv="bf16", seed=0, weights=None, apart=False,
        w_apart=False, L=None):
    """One eviction, checked in full against the reference; returns what it returned."""
    import flashattention_forward_gb300 as fa
    n = len(lens)
    most = (min(budget, max([1] + list(lens))) + page - 1) // page
    cache = sl.Cache(lens, hkv, dk, dv, page, kv, seed, extra_pages=n * most)
    L = max(1, max(lens)) if L is None else L
    g = torch.Generator().manual_seed(seed + 77)
    if weights is None:
        weights = torch.exp(2 * torch.randn((n, hkv, L), generator=g) - 3)
        weights = torch.where(weights < 0.05, torch.floor(weights * 128) / 128, weights)   # ties
    kept, new = sl.evict(weights, lens, budget, sink, recent)
    t = cache.to(DEV)
    w = weights.to(DEV)
    kw = dict(block_table=t["bt"], page_size=page, budget=budget, sink=sink, recent=recent, max_seqlen_k=max(lens),
              k_scale=t["k_scale"], v_scale=t["v_scale"])
    bt_out = cache.bt
    if apart:
        bt_out = torch.tensor(cache.free[:n * most], dtype=torch.int32).view(n, most)
        kw["block_table_out"] = bt_out.to(DEV)
    if w_apart:
        kw["weights_out"] = torch.full((n, hkv, budget + 3), 8.0, device=DEV)
    got, cu = fa.cache_evict(w, t["k"], t["v"], t["cu_k"], **kw)
    torch.cuda.synchronize()
    assert torch.equal(got.cpu(), kept)
    assert cu.cpu().tolist() == sl.cu(new).tolist()
    # the cache after the move: every byte
    for name, d in (("k", dk), ("v", dv)):
        for x, cols in ((getattr(cache, name), d), (getattr(cache, name + "_scale"), None)):
            if x is None:
                continue
            want = (sl.raw(x) if cols else x).clone()
            flat, old = want.view(-1, hkv, *([cols] if cols else [])), (sl.raw(x) if cols else x).view(-1, hkv, *([cols] if cols else []))
            for b in range(n):
                for h in range(hkv):
                    for_r = kept[b, h, :new[b]].long()
                    r = torch.arange(new[b])
                    flat[bt_out[b][r // page].long() * page + r % page, h] = old[cache.rows[b][for_r], h]
            res = t[name] if cols else t[name + "_scale"]
            assert torch.equal(bits(sl.raw(res) if cols else res), bits(want)), name
    wo = kw.get("weights_out", w)
    want = torch.zeros((n, hkv, wo.shape[2]))
    for b in range(n):
        for h in range(hkv):
            want[b, h, :new[b]] = weights[b, h][kept[b, h, :new[b]].long()]
    assert torch.equal(bits(wo), bits(want))
    if w_apart:
        assert torch.equal(bits(w), bits(weights))
    return got, cu


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("kv", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128)])
def test_types(kv, dk, dv, apart):
    run([300, 20, 0, 65, 64], 64, sink=4, recent=20, dk=dk, dv=dv, kv=kv, apart=apart, w_apart=apart, seed=dk)


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("page", [1, 2, 8, 32, 128, 1024])
def test_pages(page, apart):
    run([500, 129, 1030], 128, sink=1, recent=3, page=page, kv="e4m3", apart=apart, seed=page)


@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (7, 3, 4), (100, 0, 0), (100, 100, 0),
                                                (100, 0, 100), (100, 40, 59), (4999, 0, 0)])
def test_budgets(budget, sink, recent):
    """One key, nothing to choose, one to choose, one to drop."""
    run([5000, 101, 100, 99, 1], budget, sink, recent, hkv=3, dk=64, dv=64, seed=budget)


@pytest.mark.parametrize("n", [511, 512, 2047, 2048, 2049, 4097, 20000, 70000])
def test_lengths(n):
    run([n, n // 2], n // 3, sink=2, recent=n // 7, hkv=2, dk=64, dv=64, page=64, seed=n, w_apart=True)


def test_ties_and_special_values():
    """All equal; zeros of both signs; infinities, NaN, denormals, negatives."""
    n = 3000
    g = torch.Generator().manual_seed(0)
    rows = [torch.full((n,), 0.25), torch.zeros(n), torch.where(torch.arange(n) % 2 == 0, 0.0, -0.0),
            torch.randint(0, 3, (n,), generator=g).float(), torch.rand(n, generator=g) * 1e-41,
            -torch.rand(n, generator=g), torch.where(torch.rand(n, generator=g) < 0.9, math.nan, 1.0),
            torch.where(torch.rand(n, generator=g) < 0.5, math.inf, -math.inf)]
    w = torch.stack(rows).view(4, 2, n)
    run([n] * 4, 1000, sink=5, recent=100, dk=64, dv=64, weights=w)
    run([n] * 4, 1000, sink=5, recent=100, dk=64, dv=64, weights=w, apart=True, w_apart=True)


def test_weights_wider_than_the_sequences():
    """Entries past the keys are not chosen, and become 0."""
    run([200, 90], 64, recent=10, L=333)
    run([200, 90], 64, recent=10, L=333, apart=True, w_apart=True)


def test_strided_weights_and_cache():
    """Weights as rows of a [heads, batch, keys] buffer; K and V as two halves of one pool."""
    import flashattention_forward_gb300 as fa
    cache = sl.Cache([150, 40], 2, 64, 64, 16, "bf16", 3)
    g = torch.Generator().manual_seed(1)
    w0 = torch.rand((2, 2, 150), generator=g)
    kept, new = sl.evict(w0, [150, 40], 50, 2, 8)
    pool = torch.stack([cache.k, cache.v], 1).to(DEV)          # [N, 2, P, H, D]
    k, v = pool[:, 0], pool[:, 1]
    buf = torch.full((2, 3, 160), 4.0, device=DEV)
    w = buf[:, :2, 5:155].transpose(0, 1)
    w.copy_(w0)
    got, cu = fa.cache_evict(w, k, v, sl.cu([150, 40]).to(DEV), block_table=cache.bt.to(DEV), page_size=16, budget=50,
                             sink=2, recent=8, max_seqlen_k=150)
    torch.cuda.synchronize()
    assert torch.equal(got.cpu(), kept)
    for name, x in (("k", k), ("v", v)):
        flat, old = x.cpu().reshape(-1, 2, 64), getattr(cache, name).view(-1, 2, 64)
        for b in range(2):
            for h in range(2):
                assert torch.equal(flat[cache.rows[b][:new[b]], h], old[cache.rows[b][kept[b, h, :new[b]].long()], h])
    assert bool((buf[:, 2] == 4.0).all()) and bool((buf[..., :5] == 4.0).all()) and bool((buf[..., 155:] == 4.0).all())


def test_shared_pages_within_the_sink():
    """Sequences that share their first pages: those stay as they were."""
    import flashattention_forward_gb300 as fa
    lens = [200, 160, 64]
    cache = sl.Cache(lens, 2, 64, 64, 16, "bf16", 5, prefix=[64], groups=[0, 3])
    w0 = torch.rand((3, 2, 200), generator=torch.Generator().manual_seed(2))
    kept, new = sl.evict(w0, lens, 100, 64, 10)
    t = cache.to(DEV)
    got, _ = fa.cache_evict(w0.to(DEV), t["k"], t["v"], t["cu_k"], block_table=t["bt"], page_size=16, budget=100, sink=64,
                            recent=10, max_seqlen_k=200)
    torch.cuda.synchronize()
    assert torch.equal(got.cpu(), kept)
    flat, old = t["k"].cpu().view(-1, 2, 64), cache.k.view(-1, 2, 64)
    for b in range(3):
        for h in range(2):
            assert torch.equal(flat[cache.rows[b][:new[b]], h], old[cache.rows[b][kept[b, h, :new[b]].long()], h])


def test_captured_and_on_another_stream():
    import flashattention_forward_gb300 as fa
    cache = sl.Cache([300, 100], 2, 64, 64, 16, "bf16", 6, extra_pages=8)
    bt_out = torch.tensor(cache.free[:8], dtype=torch.int32).view(2, 4).to(DEV)
    w0 = torch.rand((2, 2, 300), generator=torch.Generator().manual_seed(3))
    kept, new = sl.evict(w0, [300, 100], 64, 1, 5)
    t, w = cache.to(DEV), w0.to(DEV)
    kw = dict(block_table=t["bt"], page_size=16, budget=64, sink=1, recent=5, max_seqlen_k=300, block_table_out=bt_out,
              weights_out=torch.empty((2, 2, 64), device=DEV), kept=torch.empty((2, 2, 64), dtype=torch.int32, device=DEV),
              cu_seqlens_k_out=torch.empty(3, dtype=torch.int32, device=DEV))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fa.cache_evict(w, t["k"], t["v"], t["cu_k"], stream=side, **kw)
    side.synchronize()
    assert torch.equal(kw["kept"].cpu(), kept)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.cache_evict(w, t["k"], t["v"], t["cu_k"], **kw)
    kw["kept"].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(kw["kept"].cpu(), kept) and kw["cu_seqlens_k_out"].tolist() == [0, 64, 128]


def test_bad_pages_and_lengths_are_flagged():
    import flashattention_forward_gb300 as fa
    for apart in (False, True):
        cache = sl.Cache([300, 100], 2, 64, 64, 16, "int8", 6, extra_pages=8)
        t = cache.to(DEV)
        t["bt"][0, 18] = 1 << 25
        t["bt"][1, 0] = -7
        out = torch.tensor(cache.free[:8], dtype=torch.int32).view(2, 4).to(DEV) if apart else None
        w = torch.rand((2, 2, 300), device=DEV)
        kw = dict(page_size=16, budget=64, recent=40, k_scale=t["k_scale"], v_scale=t["v_scale"], block_table_out=out)
        fa.cache_evict(w, t["k"], t["v"], t["cu_k"], block_table=t["bt"], max_seqlen_k=300, **kw)
        assert fa.device_error() == fa.FA_ERR_DEVICE_BOUNDS
        t = cache.to(DEV)
        kept, cu = fa.cache_evict(w[..., :200].contiguous(), t["k"], t["v"], t["cu_k"], block_table=t["bt"],
                                  max_seqlen_k=200, **kw)
        assert fa.device_error() == fa.FA_ERR_DEVICE_BOUNDS
        assert cu.tolist() == [0, 64, 128] and int(kept.max()) == 199


@pytest.mark.parametrize("w_apart", [False, True])
@pytest.mark.parametrize("lens,budget", [([9000, 8500] * 12, 3000), ([230000, 12], 120000)])
def test_long_rows_of_one_block_each(lens, budget, w_apart):
    """More rows than clusters are made for, and a row longer than eight blocks hold."""
    run(lens, budget, sink=5, recent=40, hkv=4, dk=64, dv=64, page=256, seed=len(lens), w_apart=w_apart)


def test_no_sequences_and_no_keys():
    import flashattention_forward_gb300 as fa
    z = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16, device=DEV)
    for n in (0, 3):
        kept, cu = fa.cache_evict(torch.ones((n, 2, 5), device=DEV), z, z.clone(), torch.zeros(n + 1, dtype=torch.int32, device=DEV),
                                  block_table=torch.full((n, 1), -1, dtype=torch.int32, device=DEV), page_size=16, budget=4,
                                  max_seqlen_k=0, cu_seqlens_k_out=torch.full((n + 1,), 9, dtype=torch.int32, device=DEV))
        assert cu.tolist() == [0] * (n + 1) and kept.cpu().tolist() == [[[-1] * 4] * 2] * n
