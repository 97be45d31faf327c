"""The operators around the paged decode together, as a server uses them: the
prompt's key weights, decode steps over a shared prefix that append a key and
add to the weights, an eviction, and decode steps over what was kept.  Every
step is checked against the fp64 references of serving_lib on the cache as it
stands."""
import pytest
import torch

import serving_lib as sl
from fa_testlib import LSE_TOL

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


class Server:
    """Two groups of sequences over one paged cache, on the device and, for the
    references, on the host."""
    HQ, HKV, D, PAGE, STEPS = 8, 2, 128, 16, 4
    GROUPS, PREFIX = [0, 3, 5], [160, 48]
    LENS = [260, 161, 190, 48, 300]
    BUDGET, SINK, RECENT, ROOM = 200, 160, 8, 320

    def __init__(self, kv):
        import flashattention_forward_gb300 as fa
        self.fa, self.kv = fa, kv
        lens = [n + 2 * self.STEPS for n in self.LENS]              # room for the keys to come
        self.c = sl.Cache(lens, self.HKV, self.D, self.D, self.PAGE, kv, 5, prefix=self.PREFIX, groups=self.GROUPS)
        self.lens = list(self.LENS)
        self.t = self.c.to(DEV)
        self.g = torch.Generator().manual_seed(11)
        self.w = torch.zeros((len(lens), self.HKV, self.ROOM), device=DEV)
        self.ref_w = torch.zeros((len(lens), self.HKV, self.ROOM), dtype=torch.float64)
        self.bound_w = torch.zeros_like(self.ref_w)
        self.cu_groups = torch.tensor(self.GROUPS, dtype=torch.int32, device=DEV)
        self.prefix = torch.tensor(self.PREFIX, dtype=torch.int32, device=DEV)

    def pull(self):
        """The device's cache becomes the references'."""
        for n in ("k", "v", "k_scale", "v_scale"):
            if self.t[n] is not None:
                setattr(self.c, n, self.t[n].cpu())

    def common(self):
        return dict(max_seqlen_k=max(self.lens), block_table=self.t["bt"], page_size=self.PAGE, causal=True,
                    k_scale=self.t["k_scale"])

    def cu_k(self):
        return sl.cu(self.lens).to(DEV)

    def add_weights(self, q, q_lens, lse):
        """key_weights into self.w, and the same in 64 bits."""
        self.fa.key_weights(q.to(DEV), self.t["k"], lse, sl.cu(q_lens).to(DEV), self.cu_k(), max_seqlen_q=max(q_lens),
                            weights=self.w, **self.common())
        r, b = sl.attention(q, q_lens, self.c, self.lens, causal=True, want="weights", lse=lse.cpu())
        n = r.shape[-1]
        self.ref_w[..., :n] += r
        self.bound_w[..., :n] += b
        self.bound_w += 2.0 ** -23 * self.ref_w
        sl.within(self.w, self.ref_w, self.bound_w)

    def prompt(self):
        q_lens = [n - s for n, s in zip(self.lens, (160, 0, 160, 0, 48))]      # some prefixes were computed before
        q = sl.make_q(sum(q_lens), self.HQ, self.D, 3)
        out, lse = self.fa.fwd_varlen(q.to(DEV), self.t["k"], self.t["v"], sl.cu(q_lens).to(DEV), self.cu_k(),
                                      max_seqlen_q=max(q_lens), v_scale=self.t["v_scale"], **self.common())
        # the forward's own contract: over byte caches its prompt kernels round the scaled keys to f16, 2^-11 of
        # each product (scale sum |q k| is about 7 here), which the bound for exact products leaves out
        ref = sl.attention(q, q_lens, self.c, self.lens, causal=True)
        assert float((lse.cpu().double() - ref[1]).abs().max()) <= LSE_TOL
        self.add_weights(q, q_lens, lse)

    def step(self, groups=None, prefix=None):
        """One token of each sequence: its key joins the cache, its query attends."""
        n = len(self.lens)
        for b in range(n):
            row = int(self.c.bt[b, self.lens[b] // self.PAGE]) * self.PAGE + self.lens[b] % self.PAGE
            for name in ("k", "v"):
                x, s = sl.quantize(torch.randn((self.HKV, self.D), generator=self.g), self.kv)
                sl.raw(self.t[name]).view(-1, self.HKV, self.D)[row] = sl.raw(x).to(DEV)
                if s is not None:
                    self.t[name + "_scale"].view(-1, self.HKV)[row] = s.to(DEV)
            self.lens[b] += 1
        self.pull()
        q_lens = [1] * n
        q = torch.randn((n, self.HQ, self.D), generator=self.g).to(torch.bfloat16)
        prefix = self.prefix if prefix is None else prefix
        out, lse = self.fa.fwd_shared_prefix(q.to(DEV), self.t["k"], self.t["v"], sl.cu(q_lens).to(DEV), self.cu_k(),
                                             max_seqlen_q=1, cu_groups=self.cu_groups, prefix_lens=prefix,
                                             max_prefix_len=max(self.PREFIX), v_scale=self.t["v_scale"], **self.common())
        ref = sl.attention(q, q_lens, self.c, self.lens, causal=True)
        sl.within(out, ref[0], ref[2])
        sl.within(lse, ref[1], ref[3])
        self.add_weights(q, q_lens, lse)

    def evict(self):
        """Prefix and sink stay, so the shared pages are not written."""
        before = self.w.cpu()
        want, new = sl.evict(before, self.lens, self.BUDGET, self.SINK, self.RECENT)
        kept, cu = self.fa.cache_evict(self.w, self.t["k"], self.t["v"], self.cu_k(), block_table=self.t["bt"],
                                       page_size=self.PAGE, budget=self.BUDGET, sink=self.SINK, recent=self.RECENT,
                                       max_seqlen_k=max(self.lens), k_scale=self.t["k_scale"], v_scale=self.t["v_scale"])
        assert torch.equal(kept.cpu(), want)
        assert cu.cpu().tolist() == sl.cu(new).tolist()
        old = {n: sl.raw(getattr(self.c, n)).clone() for n in ("k", "v")}
        self.pull()
        for b, n in enumerate(new):
            for h in range(self.HKV):
                j = want[b, h, :n].long()
                self.ref_w[b, h] = torch.cat([self.ref_w[b, h][j], torch.zeros(self.ROOM - n, dtype=torch.float64)])
                self.bound_w[b, h] = torch.cat([self.bound_w[b, h][j], torch.zeros(self.ROOM - n, dtype=torch.float64)])
                for name in ("k", "v"):
                    at = old[name].view(-1, self.HKV, self.D)[self.c.rows[b][j], h]
                    now = sl.raw(getattr(self.c, name)).view(-1, self.HKV, self.D)[self.c.rows[b][:n], h]
                    assert torch.equal(at.view(torch.uint8), now.view(torch.uint8))
        self.lens = new
        sl.within(self.w, self.ref_w, self.bound_w)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "int8"])
def test_prompt_decode_evict_decode(kv):
    s = Server(kv)
    s.prompt()
    for _ in range(s.STEPS):
        s.step()
    s.evict()
    assert max(s.lens) == s.BUDGET
    for _ in range(s.STEPS):
        s.step()


def test_two_captured_runs_share_a_cache():
    """A decode step and its key weights, prepared and captured twice with workspaces and outputs of
    their own, replayed in turn and at once on two streams: the results of the plain calls."""
    import flashattention_forward_gb300 as fa
    s = Server("bf16")
    n = len(s.lens)
    cu_q, cu_k = sl.cu([1] * n).to(DEV), s.cu_k()
    runs = []
    for i in range(2):
        q = sl.make_q(n, s.HQ, s.D, 20 + i).to(DEV)
        w = torch.zeros_like(s.w)
        kw = dict(max_seqlen_q=1, cu_groups=s.cu_groups, prefix_lens=s.prefix, max_prefix_len=max(s.PREFIX),
                  v_scale=None, **s.common())
        want = [x.clone() for x in fa.fwd_shared_prefix(q, s.t["k"], s.t["v"], cu_q, cu_k, **kw)]
        want_w = fa.key_weights(q, s.t["k"], want[1], cu_q, cu_k, max_seqlen_q=1, out=torch.zeros_like(s.w), **s.common())
        plan = fa.SharedPrefixPlan(q, s.t["k"], s.t["v"], cu_q, cu_k, **kw)
        out, lse = plan.run()
        weigh = fa.KeyWeightsPlan(q, s.t["k"], lse, cu_q, cu_k, max_seqlen_q=1, out=w, **s.common())
        weigh.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.run()
            weigh.run()
        runs.append((graph, (plan, weigh, q), (out, lse, w), (*want, want_w)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for x in runs:
            for t in x[2]:
                t.fill_(7.0)
        torch.cuda.synchronize()
        for stream, x in zip(streams, runs):
            with torch.cuda.stream(stream):
                x[0].replay()
        torch.cuda.synchronize()
        for x in runs:
            for got, want in zip(x[2], x[3]):
                assert torch.equal(got, want)
