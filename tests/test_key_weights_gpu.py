"""Attention weight per key against an fp64 reference (serving_lib): the rows
form (few query rows) and the tile form, cache types, pages, masks, mods."""
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


def case(q_lens, k_lens, hq=4, hkv=2, d=128, page=16, kv="bf16", seed=0, causal=True, window=0, mod="none", strided=False,
         scale=None, tail=0):
    import flashattention_forward_gb300 as fa
    cache = sl.Cache(k_lens, hkv, d, 64, page, kv, seed)
    tq = sum(q_lens)
    q = sl.make_q(tq + tail, hq, d, seed, strided)
    opts = dict(causal=causal, window=window, mod=mod, slope=0.02, cap=4.0, scale=scale)
    lse = sl.attention(q[:tq], q_lens, cache, k_lens, **opts)[1].float()
    ref = sl.attention(q[:tq], q_lens, cache, k_lens, want="weights", lse=lse, **opts)
    lse = torch.cat([lse, torch.full((hq, tail), math.nan)], 1)
    t = cache.to(DEV)
    kind = dict(none=fa.MOD_NONE, softcap=fa.MOD_SOFTCAP, alibi=fa.MOD_ALIBI)[mod]
    kw = dict(max_seqlen_q=max([1] + list(q_lens)), max_seqlen_k=max(k_lens), block_table=t["bt"], page_size=page,
              k_scale=t["k_scale"], causal=causal, window=window, score_mod=kind, alibi_slope=0.02, softcap=4.0,
              softmax_scale=scale, total_k=sum(k_lens))
    qd = q.to(DEV) if not strided else torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=DEV).copy_(q)
    return (qd, t["k"], lse.to(DEV).contiguous(), sl.cu(q_lens).to(DEV), t["cu_k"]), kw, ref


def check(args, kw, ref, **more):
    import flashattention_forward_gb300 as fa
    out = fa.key_weights(*args, **kw, **more)
    torch.cuda.synchronize()
    sl.within(out[..., :ref[0].shape[-1]], ref[0], ref[1])
    return out


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128, 192])
@pytest.mark.parametrize("page", [0, 1, 8, 16, 256])
def test_rows_form(kv, d, page):
    check(*case([1, 2, 0, 3, 1], [1, 40, 5, 130, 1000], d=d, page=page, kv=kv, hq=8, hkv=2, seed=d + page))


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128, 192])
@pytest.mark.parametrize("page", [0, 1, 16, 256])
def test_tile_form(kv, d, page):
    check(*case([130, 1, 0, 64, 257], [130, 40, 5, 300, 257], d=d, page=page, kv=kv, hq=4, hkv=2, seed=d + page))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 2), (3, 1), (5, 1), (6, 2), (7, 1), (8, 1), (16, 1), (12, 4), (48, 1),
                                    (128, 1)])
@pytest.mark.parametrize("sq", [1, 2, 70])
def test_head_layouts(hq, hkv, sq):
    check(*case([sq, 1, sq], [90, 200, max(70, sq)], hq=hq, hkv=hkv, d=64, seed=hq + sq))


@pytest.mark.parametrize("mod", ["none", "softcap", "alibi"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 60), (False, 60), (True, 1), (False, 1),
                                           (True, 2 ** 31 - 1), (False, 2 ** 31 - 1)])
@pytest.mark.parametrize("form", ["rows", "tile"])
def test_masks_and_mods(form, mod, causal, window):
    q_lens = [3, 2, 3] if form == "rows" else [200, 129, 300]
    check(*case(q_lens, [200, 600, 300], hq=4, hkv=2, causal=causal, window=window, mod=mod, kv="e4m3", seed=window % 97))


@pytest.mark.parametrize("form", ["rows", "tile"])
@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_rows_that_see_nothing(form, kv):
    """More queries than keys under a causal mask: the first rows' LSE is -inf."""
    q_lens, k_lens = ([4, 3, 2], [2, 1, 0]) if form == "rows" else ([200, 150, 30], [100, 3, 0])
    check(*case(q_lens, k_lens, kv=kv, seed=3))


@pytest.mark.parametrize("form", ["rows", "tile"])
def test_tile_edges(form):
    for nk in (127, 128, 129, 255, 256, 257, 511, 513):
        check(*case([2] if form == "rows" else [nk - 3], [nk], hq=2, hkv=1, d=64, seed=nk))


@pytest.mark.parametrize("mod,group,page", [("none", 1, 16), ("none", 3, 0), ("alibi", 1, 64), ("softcap", 2, 1)])
def test_tile_form_with_more_key_tiles_than_multiprocessors(mod, group, page):
    """Ragged lengths, so that the blocks that run take over very different key tiles of the rest: many with
    fewer query tiles than there are accumulators, some with none."""
    g = torch.Generator().manual_seed(group)
    q_lens = torch.randint(0, 260, (48,), generator=g).tolist()
    k_lens = [n + int(torch.randint(0, 400, (1,), generator=g)) * (i % 3 == 0) for i, n in enumerate(q_lens)]
    k_lens[5], k_lens[6] = 0, 3
    q_lens[5], q_lens[7], q_lens[8] = 4, 0, 600
    check(*case(q_lens, k_lens, hq=8 * group, hkv=8, d=64, page=page, mod=mod, seed=group))


@pytest.mark.parametrize("form", ["rows", "tile"])
def test_beta_out_and_strides(form):
    """Accumulation, decay, in place and apart, strided weight rows, entries past the keys."""
    import flashattention_forward_gb300 as fa
    q_lens, k_lens = ([1, 2, 0], [33, 150, 20]) if form == "rows" else ([33, 150, 0], [33, 150, 20])
    args, kw, ref = case(q_lens, k_lens, seed=1)
    L = 300
    g = torch.Generator().manual_seed(5)
    w0 = torch.rand((3, 2, L), generator=g)
    full, bound = torch.zeros((3, 2, L), dtype=torch.float64), torch.zeros((3, 2, L), dtype=torch.float64)
    full[..., :150], bound[..., :150] = ref
    for beta in (0.0, 1.0, 0.5, -2.0):
        want = beta * w0.double() + full
        tol = bound + 2.0 ** -23 * (want.abs() + abs(beta) * w0.double())
        out = torch.full((3, 2, L), 9.0, device=DEV)
        res = fa.key_weights(*args, **kw, weights=w0.to(DEV), beta=beta, out=out)
        assert res is out
        sl.within(out, want, tol)
        w = w0.to(DEV)
        assert fa.key_weights(*args, **kw, weights=w, beta=beta) is w
        sl.within(w, want, tol)
        # rows of a [heads, batch, keys] buffer, and of a wider one
        wide = torch.full((2, 4, L + 5), 3.0, device=DEV)
        view = wide[:, :3, 2:L + 2].transpose(0, 1)
        view.copy_(w0)
        fa.key_weights(*args, **kw, weights=view, beta=beta)
        sl.within(view, want, tol)
        assert bool((wide[:, 3] == 3.0).all()) and bool((wide[..., :2] == 3.0).all()) and bool((wide[..., -3:] == 3.0).all())
    # beta 0 reads nothing, no weights start from 0
    w = torch.full((3, 2, L), math.nan, device=DEV)
    fa.key_weights(*args, **kw, weights=w, beta=0.0)
    sl.within(w, full, bound)
    out = torch.full((3, 2, L), math.nan, device=DEV)
    fa.key_weights(*args, **kw, out=out)
    sl.within(out, full, bound)
    assert fa.key_weights(*args, **kw).shape == (3, 2, 150)


def test_nan_in_hidden_keys_and_foreign_rows():
    """Keys that no row sees and query rows of other sequences may hold NaN."""
    import flashattention_forward_gb300 as fa
    for q_lens, k_lens in (([2, 2], [40, 300]), ([130, 100], [200, 300])):
        args, kw, ref = case(q_lens, k_lens, causal=False, window=5, d=64, hq=3, hkv=1, tail=4, seed=6)
        # window 5, not causal: keys more than 4 left of the first row are hidden
        hid = k_lens[1] - q_lens[1] - 5
        cache = args[1]
        rows = kw["block_table"][1].long()
        j = torch.arange(hid, device=DEV)
        cache.view(-1, 1, 64)[rows[j // 16] * 16 + j % 16] = math.nan
        args[0][sum(q_lens):] = math.nan
        out = fa.key_weights(*args, **kw)
        sl.within(out, ref[0], ref[1])


@pytest.mark.parametrize("form", ["rows", "tile"])
def test_other_scales_and_strided_q(form):
    q_lens = [2, 1] if form == "rows" else [100, 30]
    for scale in (-0.2, 0.0, 0.5):
        check(*case(q_lens, [120, 300], scale=scale, strided=True, d=64, seed=4))


@pytest.mark.parametrize("form", ["rows", "tile"])
def test_plan_graph_and_repeats(form):
    import flashattention_forward_gb300 as fa
    q_lens = [1, 2] if form == "rows" else [300, 130]
    args, kw, ref = case(q_lens, [300, 700], hq=8, hkv=2, seed=2)
    a = check(args, kw, ref)
    plan = fa.KeyWeightsPlan(*args, **kw)
    assert torch.equal(plan.run(), a)
    g = torch.cuda.CUDAGraph()
    out = plan.run()
    with torch.cuda.graph(g):
        plan.run()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = fa.key_weights(*args, **kw, stream=side)
    side.synchronize()
    assert torch.equal(a, b)


def test_sums_are_the_number_of_rows():
    """Each visible row's weights sum to one per head."""
    args, kw, ref = case([1000, 500], [1000, 900], hq=4, hkv=2, seed=7)
    out = check(args, kw, ref)
    want = torch.tensor([1000.0, 500.0])[:, None] * 2
    assert float((out.sum(-1).cpu() / want - 1).abs().max()) < 1e-4


def test_lengths_beyond_the_bounds_and_bad_pages_are_flagged():
    import flashattention_forward_gb300 as fa
    for q_lens in ([1, 1], [100, 40]):
        args, kw, ref = case(q_lens, [100, 40])
        kw["max_seqlen_k"] = 60
        fa.key_weights(*args, **kw, out=torch.zeros((2, 2, 60), device=DEV))
        assert fa.device_error() == fa.FA_ERR_DEVICE_BOUNDS
        kw["max_seqlen_k"] = 100
        kw["block_table"][0, 2] = 1 << 24
        out = fa.key_weights(*args, **kw)
        assert fa.device_error() == fa.FA_ERR_DEVICE_BOUNDS
        sl.within(out[1], ref[0][1], ref[1][1])


@pytest.mark.parametrize("form", ["rows", "tile"])
@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_scales_from_zero_to_large(form, kv):
    """Key scales of 0 (whatever the bytes), far below and far above the others."""
    import flashattention_forward_gb300 as fa
    q_lens, k_lens = ([2], [260]) if form == "rows" else ([200], [260])
    cache = sl.Cache(k_lens, 2, 64, 64, 16, kv, 5)
    q = sl.make_q(q_lens[0], 4, 64, 5)
    f = torch.ones(260, 2)
    f[::7], f[1::7], f[2::7], f[3::7] = 0.0, 1e-38, 1e-6, 8.0
    cache.k_scale.view(-1, 2)[cache.rows[0]] *= f
    opts = dict(causal=True)
    lse = sl.attention(q, q_lens, cache, k_lens, **opts)[1].float()
    ref = sl.attention(q, q_lens, cache, k_lens, want="weights", lse=lse, **opts)
    t = cache.to(DEV)
    check((q.to(DEV), t["k"], lse.to(DEV), sl.cu(q_lens).to(DEV), t["cu_k"]),
          dict(max_seqlen_q=q_lens[0], max_seqlen_k=260, block_table=t["bt"], page_size=16, k_scale=t["k_scale"],
               causal=True), ref)


@pytest.mark.parametrize("form", ["rows", "tile"])
def test_query_rows_outside_q_are_flagged_and_add_nothing(form):
    import flashattention_forward_gb300 as fa
    args, kw, ref = case([1, 2] if form == "rows" else [100, 40], [100, 40])
    args[3][2] = 1 << 20
    kw["max_seqlen_q"] = 2 if form == "rows" else 100
    out = fa.key_weights(*args, **kw)
    assert fa.device_error() == fa.FA_ERR_DEVICE_BOUNDS
    sl.within(out[0], ref[0][0], ref[1][0])
    assert bool((out[1] == 0).all())


def test_no_queries_and_no_keys():
    """Without query rows the old weights decay; without sequences or entries nothing happens."""
    import flashattention_forward_gb300 as fa
    k = torch.zeros((1, 16, 2, 64), dtype=torch.bfloat16, device=DEV)
    q, lse = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=DEV), torch.zeros((4, 0), device=DEV)
    for n, L in ((2, 40), (2, 0), (0, 40)):
        w = torch.rand((n, 2, L), device=DEV)
        old = w.clone()
        cu_k = torch.arange(0, 3 * (n + 1), 3, dtype=torch.int32, device=DEV) if L else torch.zeros(n + 1, dtype=torch.int32, device=DEV)
        fa.key_weights(q, k, lse, torch.zeros(n + 1, dtype=torch.int32, device=DEV), cu_k, max_seqlen_q=0,
                       max_seqlen_k=min(L, 3), block_table=torch.zeros((n, 1), dtype=torch.int32, device=DEV), page_size=16,
                       weights=w, beta=0.5)
        assert torch.equal(w, 0.5 * old)
