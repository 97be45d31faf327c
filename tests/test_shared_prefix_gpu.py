"""Decode of a batch whose sequences share prefixes, against an fp64 reference
(serving_lib): cache types, head layouts, page sizes, masks, ragged groups."""
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


def case(groups=(0, 3), prefix=(64,), suffix=(5, 17, 1), q_lens=None, hq=4, hkv=2, d=128, page=16, kv="bf16", seed=0,
         causal=True, window=0, mod="none", prefix_splits=None, num_splits=None, strided=False, tail=0, scale=None,
         k_lens=None):
    import flashattention_forward_gb300 as fa
    groups, prefix, suffix = list(groups), list(prefix), list(suffix)
    whole = [p // page * page for p in prefix]
    owner = [x for x in range(len(prefix)) for _ in range(groups[x], groups[x + 1])]
    if k_lens is None:
        k_lens = [whole[owner[b]] + suffix[b] for b in range(len(suffix))]
    q_lens = [1] * len(k_lens) if q_lens is None else list(q_lens)
    cache = sl.Cache(k_lens, hkv, d, d, page, kv, seed, prefix=whole, groups=groups)
    tq = sum(q_lens)
    q = sl.make_q(tq + tail, hq, d, seed, strided)
    t = cache.to(DEV)
    kind = dict(none=fa.MOD_NONE, softcap=fa.MOD_SOFTCAP, alibi=fa.MOD_ALIBI)[mod]
    kw = dict(max_seqlen_q=max(q_lens), max_seqlen_k=max(k_lens), block_table=t["bt"], page_size=page,
              cu_groups=torch.tensor(groups, dtype=torch.int32, device=DEV),
              prefix_lens=torch.tensor(prefix, dtype=torch.int32, device=DEV), max_prefix_len=max(prefix),
              total_k=sum(k_lens), k_scale=t["k_scale"], v_scale=t["v_scale"], causal=causal, window=window,
              score_mod=kind, alibi_slope=0.05, softcap=3.0, prefix_splits=prefix_splits, num_splits=num_splits,
              softmax_scale=scale)
    args = (q.to(DEV) if not strided else sl.make_q(tq + tail, hq, d, seed, True).to(DEV), t["k"], t["v"],
            sl.cu(q_lens).to(DEV), t["cu_k"])
    ref = sl.attention(q[:tq], q_lens, cache, k_lens, causal=causal, window=window, mod=mod, slope=0.05, cap=3.0,
                       scale=scale)
    return args, kw, ref


def check(args, kw, ref, **more):
    import flashattention_forward_gb300 as fa
    out, lse = fa.fwd_shared_prefix(*args, **kw, **more)
    torch.cuda.synchronize()
    n = ref[0].shape[0]
    sl.within(out[:n], ref[0], ref[2])
    sl.within(lse[:, :n], ref[1], ref[3])
    return out, lse


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [1, 4, 8, 16, 64, 256])
def test_types_and_pages(kv, d, page):
    check(*case(groups=(0, 3, 5), prefix=(520, 300), suffix=(5, 70, 1, 33, 129), d=d, page=page, kv=kv, hq=8, hkv=2,
                seed=page + d))


@pytest.mark.parametrize("hq,hkv,sq", [(1, 1, 1), (16, 1, 1), (3, 1, 3), (6, 2, 2), (7, 1, 2), (8, 8, 4), (15, 3, 3),
                                       (12, 4, 5)])
def test_head_layouts(hq, hkv, sq):
    """Groups of 1 to 16 heads, also ones that do not divide a tile's rows."""
    check(*case(groups=(0, 4), prefix=(200,), suffix=(9, 30, 6, 64), q_lens=(sq, 1, sq, 0), hq=hq, hkv=hkv, seed=hq))


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("n", [31, 33, 64, 200])
def test_many_sequences(n, kv):
    """Several row tiles per kv head, the last one part full."""
    check(*case(groups=(0, n), prefix=(300,), suffix=[1 + (7 * b) % 40 for b in range(n)], hq=8, hkv=2, kv=kv, seed=n))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("mod", ["none", "softcap", "alibi"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 90), (False, 90), (True, 1), (False, 1)])
def test_masks_and_mods(mod, causal, window, kv):
    check(*case(groups=(0, 2, 4), prefix=(256, 144), suffix=(3, 40, 7, 100), q_lens=(3, 2, 1, 3), hq=8, hkv=2, kv=kv,
                causal=causal, window=window, mod=mod, seed=window + 3))


def test_rows_that_end_inside_the_prefix():
    """Sequences shorter than the shared pages: each row keeps its own limit,
    one sees nothing at all."""
    check(*case(groups=(0, 4), prefix=(256,), suffix=(0,) * 4, k_lens=(256, 100, 3, 0), q_lens=(2, 2, 4, 2), seed=5))


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_empty_and_single_groups(kv):
    """Empty groups, groups of one, prefixes of 0 and of less than a page, idle
    slots, sequences without a key of their own."""
    check(*case(groups=(0, 0, 1, 3, 3, 5), prefix=(64, 128, 0, 64, 15), suffix=(0, 5, 1, 200, 64),
                q_lens=(1, 1, 0, 1, 1), causal=False, kv=kv, seed=9))


def test_many_groups():
    """More groups than a warp has lanes."""
    n = 70
    check(*case(groups=list(range(0, 2 * n + 1, 2)), prefix=[16 * (x % 5) for x in range(n)],
                suffix=[1 + x % 9 for x in range(2 * n)], seed=4, d=64))


@pytest.mark.parametrize("ps,ns", [(1, 1), (2, 3), (5, 1), (40, 33), (64, 64)])
def test_split_counts(ps, ns):
    """More splits than key tiles leaves some empty."""
    check(*case(prefix=(640,), suffix=(100, 300, 1), prefix_splits=ps, num_splits=ns, hq=8, hkv=2, seed=ps))


def test_host_bounds_only_size_the_work():
    """A prefix longer than max_prefix_len, and own keys beyond what it implies, are attended in full."""
    args, kw, ref = case(prefix=(640,), suffix=(100, 300, 1), num_splits=2)
    kw["max_prefix_len"] = 16
    check(args, kw, ref)
    kw["max_prefix_len"] = 640 + 290
    check(args, kw, ref)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 0.7])
def test_other_scales(scale):
    check(*case(scale=scale, suffix=(50, 60, 70), seed=2))


@pytest.mark.parametrize("size", [1e-3, 1.0, 300.0])
@pytest.mark.parametrize("kv", ["bf16", "e4m3", "int8"])
def test_magnitude_of_v(kv, size):
    """The scaled weights keep their precision whatever the magnitude of V."""
    args, kw, _ = case(groups=(0, 3), prefix=(256,), suffix=(9, 1, 40), kv=kv, seed=8)
    cache = sl.Cache([265, 257, 296], 2, 128, 128, 16, kv, 8, prefix=[256], groups=[0, 3])
    if kv == "bf16":
        args[2].mul_(size)
        cache.v.mul_(size)
    else:
        kw["v_scale"].mul_(size)
        cache.v_scale.mul_(size)
    ref = sl.attention(args[0].cpu(), [1, 1, 1], cache, cache.lens, causal=True)
    import flashattention_forward_gb300 as fa
    out, lse = fa.fwd_shared_prefix(*args, **kw)
    sl.within(out, ref[0], ref[2])
    sl.within(lse, ref[1], ref[3])


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_scales_of_very_different_size(kv):
    """V scales that grow along the prefix, and tiles whose V is all zero."""
    args, kw, _ = case(groups=(0, 3), prefix=(512,), suffix=(9, 1, 40), kv=kv, seed=8, prefix_splits=1)
    cache = sl.Cache([521, 513, 552], 2, 128, 128, 16, kv, 8, prefix=[512], groups=[0, 3])
    f = torch.ones(512)
    f[:128], f[128:256], f[384:] = 0.0, 1e-4, 50.0
    for vs in (cache.v_scale, kw["v_scale"]):
        vs.view(-1, 2)[cache.rows[0][:512].to(vs.device)] *= f.to(vs.device)[:, None]
    ref = sl.attention(args[0].cpu(), [1, 1, 1], cache, cache.lens, causal=True)
    check(args, kw, ref)


def test_strided_q_and_padded_rows():
    """q as a view of a fused projection; rows behind the last sequence stay as they were."""
    args, kw, ref = case(strided=True, tail=6, suffix=(9, 20, 3), q_lens=(2, 1, 3))
    out = torch.full((12, 4, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((4, 12), 6.0, device=DEV)
    check(args, kw, ref, out=out, lse=lse)
    assert bool((out[6:] == 5.0).all()) and bool((lse[:, 6:] == 6.0).all())


def test_matches_the_plain_decode():
    """The same call through fwd_varlen (no sharing) agrees to rounding."""
    import flashattention_forward_gb300 as fa
    args, kw, ref = case(groups=(0, 5, 8), prefix=(1024, 512), suffix=[1, 50, 100, 3, 7, 64, 65, 300], hq=32, hkv=8)
    out, lse = check(args, kw, ref)
    for n in ("cu_groups", "prefix_lens", "max_prefix_len", "prefix_splits"):
        kw.pop(n)
    o2, l2 = fa.fwd_varlen(*args, **kw)
    torch.cuda.synchronize()
    sl.within(o2, ref[0], ref[2])
    assert float((lse - l2).abs().max()) < 1e-4


def test_plan_graph_streams_and_repeats():
    """Plan, captured graph, another stream, one stream after another: the same
    bits; new lengths are read at each run; no lse."""
    import flashattention_forward_gb300 as fa
    args, kw, ref = case(groups=(0, 3), prefix=(400,), suffix=(30, 90, 1), hq=8, hkv=2)
    out, lse = check(args, kw, ref)
    plan = fa.SharedPrefixPlan(*args, **kw)
    o, l = plan.run()
    assert torch.equal(o, out) and torch.equal(l, lse)
    o.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan.run(stream=side)
    side.synchronize()
    assert torch.equal(o, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.run()
    o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out)
    o3, l3 = fa.fwd_shared_prefix(*args, **kw, stream=side)
    side.synchronize()
    assert torch.equal(o3, out) and torch.equal(l3, lse)
    o4, l4 = fa.fwd_shared_prefix(*args, **kw, return_lse=False)
    assert l4 is None and torch.equal(o4, out)
    # one key less in the last sequence's own part, prefix of the group halved: same plan
    kw["prefix_lens"].fill_(200)
    plan.run()
    torch.cuda.synchronize()
    sl.within(o, ref[0], ref[2])


def test_bad_pages_are_flagged_not_followed():
    """Page ids outside the pool in the prefix and behind it: an error word, no fault."""
    import flashattention_forward_gb300 as fa
    for page, kv in ((16, "bf16"), (4, "bf16"), (16, "e4m3"), (4, "int8")):
        args, kw, _ = case(page=page, kv=kv, prefix=(64,), suffix=(50, 20, 10))
        kw["block_table"][0, 1] = 1 << 20
        kw["block_table"][1, 64 // page] = -5
        fa.fwd_shared_prefix(*args, **kw)
        assert fa.device_error() == fa.FA_ERR_DEVICE_BOUNDS


def test_groups_that_leave_sequences_out_are_flagged():
    import flashattention_forward_gb300 as fa
    args, kw, _ = case()
    kw["cu_groups"][1] = 2
    fa.fwd_shared_prefix(*args, **kw)
    assert fa.device_error() == fa.FA_ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_query_rows_outside_q_are_flagged_and_not_written(kv):
    """cu_seqlens_q that runs past T_q: the sequences before keep their results."""
    import flashattention_forward_gb300 as fa
    args, kw, ref = case(groups=(0, 2, 4), prefix=(300, 64), suffix=(9, 30, 6, 64), kv=kv)
    args[3][4] = 9
    out = torch.full((6, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((4, 6), 7.0, device=DEV)
    fa.fwd_shared_prefix(*args, **kw, out=out[:4], lse=lse.view(-1)[:16].view(4, 4))
    assert fa.device_error() == fa.FA_ERR_DEVICE_BOUNDS
    sl.within(out[:2], ref[0][:2], ref[2][:2])
    assert bool((out[4:] == 7).all()) and bool((lse.view(-1)[16:] == 7).all())
