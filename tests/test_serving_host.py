"""Host-only checks of the shared-prefix, key-weight and eviction entries:
malformed calls are refused with a status and a message before any CUDA call."""
import ctypes
import math

import pytest
import torch

import flashattention_forward_gb300 as fa
from flashattention_forward_gb300 import build as fa_build

INV, UNS, OVF = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_OVERFLOW
BASE = 1 << 24   # never dereferenced: every call here is refused


@pytest.fixture(scope="module")
def L():
    fa_build.build()
    return fa.lib()


def T(slot, dtype, shape, stride=None, offset=0):
    t = fa.Tensor()
    t.data = BASE * (slot + 1) + offset
    t.dtype = dtype
    t.ndim = len(shape)
    if stride is None:
        stride, s = [], 1
        for x in reversed(shape):
            stride.insert(0, s)
            s *= x
    t.shape[:len(shape)] = shape
    t.stride[:len(shape)] = stride
    return t


def ref(x):
    return None if x is None else ctypes.byref(x)


def launch(**over):
    d = dict(num_seqs=3, max_seqlen_q=2, max_seqlen_k=100, num_splits=1, total_q=5, total_k=0, workspace=BASE * 90,
             workspace_bytes=1 << 23, flags=0)
    d.update(over)
    return fa.Launch(**d)


def prefix(**over):
    d = dict(cu_groups=BASE * 80, lens=BASE * 81, num_groups=1, max_len=64, num_splits=2)
    d.update(over)
    return fa.SharedPrefix(**d)


def call_prefix(L, plan=False, **over):
    a = dict(q=T(0, fa.FA_BF16, [5, 4, 128]), k=T(1, fa.FA_BF16, [20, 16, 2, 128]), v=T(2, fa.FA_BF16, [20, 16, 2, 128]),
             bt=T(3, fa.FA_I32, [3, 7]), cq=T(4, fa.FA_I32, [4]), ck=T(5, fa.FA_I32, [4]), ks=None, vs=None,
             out=T(6, fa.FA_BF16, [5, 4, 128]), lse=T(7, fa.FA_F32, [4, 5]), scale=0.1, causal=1, window=0, mod=None,
             prefix=prefix(), page=16, launch=launch())
    a.update(over)
    args = [ref(a[n]) for n in ("q", "k", "v", "bt", "cq", "ck", "ks", "vs", "out", "lse")] + \
        [a["scale"], a["causal"], a["window"], ref(a["mod"]), ref(a["prefix"]), a["page"], ref(a["launch"])]
    if plan:
        h = ctypes.c_void_p(1)
        st = L.fa_shared_prefix_plan_create(*args, ctypes.byref(h))
        assert not h.value
    else:
        st = L.fa_fwd_shared_prefix(*args, None)
    return st, L.fa_last_error().decode()


E4 = dict(k=T(1, fa.FA_E4M3, [20, 16, 2, 128]), v=T(2, fa.FA_E4M3, [20, 16, 2, 128]))

PREFIX_CASES = [
    (dict(q=None), INV, "q is NULL"),
    (dict(q=T(0, fa.FA_F32, [5, 4, 128])), INV, "dtype"),
    (dict(q=T(0, fa.FA_BF16, [6, 4, 128])), INV, "total_q"),
    (dict(q=T(0, fa.FA_BF16, [5, 4, 128], [516, 129, 1])), INV, "16 bytes"),
    (dict(q=T(0, fa.FA_BF16, [5, 4, 128], offset=8)), INV, "aligned"),
    (dict(q=T(0, fa.FA_BF16, [5, 3, 128])), INV, "multiple of Hkv"),
    (dict(bt=None), UNS, "paged"),
    (dict(bt=T(3, fa.FA_I32, [2, 7])), INV, "rows"),
    (dict(bt=T(3, fa.FA_I32, [3, 6])), INV, "block_table holds 96"),
    (dict(bt=T(3, fa.FA_F32, [3, 7])), INV, "dtype"),
    (dict(k=None), INV, "k_cache is NULL"),
    (dict(k=T(1, fa.FA_F32, [20, 16, 2, 128])), INV, "bf16, e4m3 or int8"),
    (dict(k=T(1, fa.FA_BF16, [20, 16, 2, 64])), INV, "head dim"),
    (dict(k=T(1, fa.FA_E4M3, [20, 2, 8, 16, 16]), v=T(2, fa.FA_E4M3, [20, 2, 1, 128, 16])), UNS, "5-D"),
    (dict(k=T(1, fa.FA_BF16, [21, 16, 2, 128])), INV, "disagree"),
    (dict(v=T(2, fa.FA_E4M3, [20, 16, 2, 128])), INV, "types differ"),
    (dict(k=T(1, fa.FA_BF16, [20, 16, 2, 128], offset=2)), INV, "aligned"),
    (dict(page=32), INV, "page holds 16"),
    (dict(page=12), UNS, "powers of two"),
    (dict(page=0), UNS, "powers of two"),
    (dict(page=2048), UNS, "1 to 1024"),
    (E4, INV, "need k_scale"),
    (dict(ks=T(8, fa.FA_F32, [20, 16, 2])), INV, "only valid with"),
    (dict(E4, ks=T(8, fa.FA_F32, [20, 16, 1]), vs=T(9, fa.FA_F32, [20, 16, 2])), INV, "k_scale must be"),
    (dict(q=T(0, fa.FA_BF16, [5, 4, 192]), k=T(1, fa.FA_BF16, [20, 16, 2, 192])), UNS, "Dk = Dv"),
    (dict(cq=T(4, fa.FA_I32, [3])), INV, "cu_seqlens_q"),
    (dict(out=T(6, fa.FA_F32, [5, 4, 128])), INV, "dtype"),
    (dict(out=T(6, fa.FA_BF16, [5, 4, 64])), INV, "out must be"),
    (dict(out=T(0, fa.FA_BF16, [5, 4, 128])), INV, "alias"),
    (dict(lse=T(7, fa.FA_F32, [5, 4])), INV, "lse must be"),
    (dict(scale=math.inf), INV, "softmax_scale"),
    (dict(mod=fa.ScoreMod(kind=2, softcap=0.0)), INV, "softcap"),
    (dict(mod=fa.ScoreMod(kind=5)), INV, "score_mod"),
    (dict(prefix=None), INV, "prefix is NULL"),
    (dict(prefix=prefix(num_groups=0)), INV, "num_groups"),
    (dict(prefix=prefix(num_splits=0)), INV, "num_splits"),
    (dict(prefix=prefix(max_len=-1)), INV, "max_len"),
    (dict(prefix=prefix(cu_groups=None)), INV, "cu_groups"),
    (dict(prefix=prefix(num_groups=70000)), UNS, "tiles"),
    (dict(launch=None), INV, "launch is NULL"),
    (dict(launch=launch(num_splits=0)), INV, "num_splits"),
    (dict(launch=launch(num_splits=5000)), UNS, "splits"),
    (dict(launch=launch(flags=1)), INV, "flags"),
    (dict(launch=launch(max_seqlen_q=9)), UNS, "Hq/Hkv <= 16"),
    (dict(launch=launch(max_seqlen_q=0)), INV, "max_seqlen_q"),
    (dict(launch=launch(max_seqlen_k=1 << 30)), OVF, "2^30"),
    (dict(launch=launch(workspace=None)), INV, "workspace"),
    (dict(launch=launch(workspace_bytes=100)), INV, "workspace"),
    (dict(launch=launch(workspace=BASE * 90 + 16)), INV, "256-byte"),
]


@pytest.mark.parametrize("over,status,words", PREFIX_CASES)
def test_shared_prefix_refusals(L, over, status, words):
    st, msg = call_prefix(L, **over)
    assert st == status and words in msg, (st, msg)
    st, msg = call_prefix(L, plan=True, **over)
    assert st == status and words in msg


def test_shared_prefix_sizes(L):
    x, p = launch(num_splits=3, total_q=10), prefix(num_splits=5)
    assert fa.shared_prefix_workspace_bytes(x, p, 32, 128) == 8 * 10 * 32 * 128 * 4 + 8 * 32 * 10 * 4
    assert fa.shared_prefix_workspace_bytes(launch(total_q=0), p, 32, 128) == 0
    assert L.fa_shared_prefix_workspace_bytes(None, ctypes.byref(p), 32, 128) == 0
    assert fa.shared_prefix_default_splits(64, 1, 100, 32, 8) == 1           # a single key tile
    assert fa.shared_prefix_default_splits(64, 1, 0, 32, 8) == 1
    assert 1 <= fa.shared_prefix_default_splits(64, 1, 8192, 32, 8) <= 64
    assert fa.shared_prefix_default_splits(1 << 20, 1, 8192, 32, 8) == 1
    assert fa.shared_prefix_default_own_splits(4, 0, 0, 8) == 1
    assert fa.shared_prefix_default_own_splits(4, 64, 256, 8) == 1
    assert fa.shared_prefix_default_own_splits(4, 65, 256, 8) == 2
    assert 2 <= fa.shared_prefix_default_own_splits(64, 8192, 64 * 4000, 8) <= 64


def call_weights(L, plan=False, **over):
    a = dict(q=T(0, fa.FA_BF16, [5, 4, 128]), k=T(1, fa.FA_BF16, [20, 16, 2, 128]), bt=T(3, fa.FA_I32, [3, 7]),
             cq=T(4, fa.FA_I32, [4]), ck=T(5, fa.FA_I32, [4]), ks=None, lse=T(7, fa.FA_F32, [4, 5]),
             w=T(10, fa.FA_F32, [3, 2, 100]), beta=1.0, out=T(11, fa.FA_F32, [3, 2, 100]), scale=0.1, causal=1, window=0,
             mod=None, page=16, launch=launch())
    a.update(over)
    args = [ref(a[n]) for n in ("q", "k", "bt", "cq", "ck", "ks", "lse", "w")] + \
        [a["beta"], ref(a["out"]), a["scale"], a["causal"], a["window"], ref(a["mod"]), a["page"], ref(a["launch"])]
    if plan:
        h = ctypes.c_void_p(1)
        st = L.fa_key_weights_plan_create(*args, ctypes.byref(h))
        assert not h.value
    else:
        st = L.fa_key_weights(*args, None)
    return st, L.fa_last_error().decode()


WEIGHT_CASES = [
    (dict(q=T(0, fa.FA_E4M3, [5, 4, 128])), INV, "dtype"),
    (dict(k=T(1, fa.FA_BF16, [20, 16, 2, 96]), q=T(0, fa.FA_BF16, [5, 4, 96])), UNS, "not compiled"),
    (dict(q=T(0, fa.FA_BF16, [5, 258, 128]), lse=T(7, fa.FA_F32, [258, 5])), UNS, "<= 128"),
    (dict(bt=None), INV, "3"),
    (dict(bt=None, k=T(1, fa.FA_BF16, [50, 2, 128]), launch=launch(total_k=60)), INV, "fewer rows"),
    (dict(k=T(1, fa.FA_I8, [20, 16, 2, 128])), INV, "need k_scale"),
    (dict(lse=None), INV, "lse is NULL"),
    (dict(lse=T(7, fa.FA_F32, [4, 5], [6, 1])), INV, "contiguous"),
    (dict(out=None), INV, "out is NULL"),
    (dict(out=T(11, fa.FA_F32, [3, 2, 99]), w=T(10, fa.FA_F32, [3, 2, 99])), INV, "max_seqlen_k"),
    (dict(out=T(11, fa.FA_F32, [3, 4, 100])), INV, "Hkv"),
    (dict(out=T(11, fa.FA_F32, [3, 2, 100], [200, 100, 2])), INV, "contiguous last dim"),
    (dict(out=T(11, fa.FA_F32, [3, 2, 100], [0, 100, 1])), INV, "overlap each other"),
    (dict(out=T(11, fa.FA_F32, [3, 2, 100], [200, 60, 1])), INV, "overlap each other"),
    (dict(w=T(10, fa.FA_F32, [3, 2, 101])), INV, "same shape"),
    (dict(w=T(11, fa.FA_F32, [3, 2, 100], offset=4)), INV, "not overlap"),
    (dict(w=T(11, fa.FA_F32, [3, 2, 100], [100, 300, 1])), INV, "not overlap"),
    (dict(out=T(7, fa.FA_F32, [3, 2, 100])), INV, "alias"),
    (dict(beta=math.nan), INV, "beta"),
    (dict(scale=math.nan), INV, "softmax_scale"),
    (dict(mod=fa.ScoreMod(kind=1, alibi_slope=math.inf)), INV, "alibi"),
    (dict(launch=launch(max_seqlen_q=0)), INV, "max_seqlen_q"),
    (dict(launch=launch(num_seqs=70000)), UNS, "65535"),
    (dict(launch=launch(max_seqlen_k=-1)), INV, "negative"),
]


@pytest.mark.parametrize("over,status,words", WEIGHT_CASES)
def test_key_weights_refusals(L, over, status, words):
    st, msg = call_weights(L, **over)
    assert st == status and words in msg, (st, msg)
    st, msg = call_weights(L, plan=True, **over)
    assert st == status and words in msg


def call_evict(L, **over):
    a = dict(w=T(10, fa.FA_F32, [3, 2, 100]), wo=None, k=T(1, fa.FA_BF16, [20, 16, 2, 128]),
             v=T(2, fa.FA_BF16, [20, 16, 2, 128]), ks=None, vs=None, bt=T(3, fa.FA_I32, [3, 7]), bto=None,
             ck=T(5, fa.FA_I32, [4]), cko=T(12, fa.FA_I32, [4]), kept=T(13, fa.FA_I32, [3, 2, 50]), budget=50, sink=2,
             recent=10, page=16, launch=launch())
    a.update(over)
    st = L.fa_cache_evict(*[ref(a[n]) for n in ("w", "wo", "k", "v", "ks", "vs", "bt", "bto", "ck", "cko", "kept")],
                          a["budget"], a["sink"], a["recent"], a["page"], ref(a["launch"]), None)
    return st, L.fa_last_error().decode()


EVICT_CASES = [
    (dict(w=None), INV, "weights is NULL"),
    (dict(w=T(10, fa.FA_F32, [3, 2, 99])), INV, "max_seqlen_k"),
    (dict(w=T(10, fa.FA_F32, [3, 2, 100], [0, 100, 1])), INV, "overlap each other"),
    (dict(wo=T(14, fa.FA_F32, [3, 2, 49])), INV, "may stay"),
    (dict(wo=T(10, fa.FA_F32, [3, 2, 100], offset=64)), INV, "not overlap"),
    (dict(bt=None), UNS, "paged"),
    (dict(bto=T(15, fa.FA_I32, [3, 3])), INV, "block_table_out holds 48"),
    (dict(bto=T(15, fa.FA_I32, [2, 4])), INV, "rows"),
    (dict(v=T(2, fa.FA_BF16, [20, 16, 2, 64])), UNS, "not compiled"),
    (dict(v=T(2, fa.FA_I8, [20, 16, 2, 128])), INV, "types differ"),
    (dict(v=T(1, fa.FA_BF16, [20, 16, 2, 128])), INV, "must not overlap each other"),
    (dict(E4), INV, "need k_scale"),
    (dict(E4, ks=T(8, fa.FA_F32, [20, 16, 2]), vs=T(8, fa.FA_F32, [20, 16, 2])), INV, "must not overlap each other"),
    (dict(kept=T(13, fa.FA_I32, [3, 2, 49])), INV, "kept"),
    (dict(kept=T(13, fa.FA_F32, [3, 2, 50])), INV, "dtype"),
    (dict(cko=None), INV, "cu_seqlens_k_out is NULL"),
    (dict(cko=T(5, fa.FA_I32, [4])), INV, "overlap"),
    (dict(kept=T(10, fa.FA_I32, [3, 2, 50])), INV, "overlap"),
    (dict(budget=0), INV, "budget"),
    (dict(sink=-1), INV, "sink"),
    (dict(recent=-1), INV, "recent"),
    (dict(sink=30, recent=21), INV, "sink + recent"),
    (dict(page=8), INV, "page holds 16"),
    (dict(launch=None), INV, "launch is NULL"),
    (dict(launch=launch(max_seqlen_k=113)), INV, "block_table holds 112"),
    (dict(launch=launch(num_seqs=70000)), UNS, "65535"),
]


@pytest.mark.parametrize("over,status,words", EVICT_CASES)
def test_cache_evict_refusals(L, over, status, words):
    st, msg = call_evict(L, **over)
    assert st == status and words in msg, (st, msg)


def test_plan_is_required(L):
    assert L.fa_shared_prefix_plan_create(*[None] * 10, 0.1, 1, 0, None, None, 16, None, None) == INV
    assert L.fa_key_weights_plan_create(*[None] * 8, 1.0, None, 0.1, 1, 0, None, 16, None, None) == INV


def test_python_calls_want_cuda_tensors_of_one_device():
    z = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        fa.fwd_shared_prefix(z, z, z, i, i)
    with pytest.raises(ValueError, match="CUDA device"):
        fa.key_weights(z, z, z, i, i)
    with pytest.raises(ValueError, match="CUDA device"):
        fa.cache_evict(torch.zeros(1, 1, 4), z, z, i, block_table=i, page_size=16, budget=1, max_seqlen_k=4)
