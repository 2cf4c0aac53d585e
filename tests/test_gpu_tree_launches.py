"""How the calls over trees are launched: one behind the other with programmatic dependent launches, eager and in a graph;
on a stream that is not the current one; two streams at a time.  Results are those of the plain calls, bit for bit."""
import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

import _layer_ref as layer_ref
import _tree_ref as ref

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32
H, D, KW, WIDE = 2, 64, 4, 16          # heads of everything, their width, taps, query heads of the wide attention


@pytest.fixture(scope="module")
def libs(built_libs):
    return {F32: kda.KdaLibrary(F32), F16: kda.KdaLibrary(F16)}


class Chain:
    """Steps over the same trees whose calls each take what the call before left: convolutions, recurrence, append, attention by
    either kernel and again on the first's output, acceptance; the next step goes on from the accepted nodes."""

    def __init__(self, lib, pool_dtype, shapes, ctx, steps, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.lib, self.steps = lib, steps
        pars = [ref.parents(t, k, i) for i, (t, k) in enumerate(shapes)]
        lens = [len(p) for p in pars]
        self.n, self.total, self.max_t = len(lens), sum(lens), max(lens)
        cu = [0]
        for t in lens:
            cu.append(cu[-1] + t)
        self.cu, self.tree = torch.tensor(cu, dtype=I32, device="cuda"), ref.masks(pars)
        n, total = self.n, self.total
        self.pool0 = (0.3 * r(n * self.max_t, H, D, D)).to(pool_dtype).cuda()
        self.table = torch.arange(n * self.max_t, dtype=I32, device="cuda").view(n, -1)
        cache = layer_ref.Cache([c + t for c, t in zip(ctx, lens)], H, D, 32, g)
        self.pages0, self.ptab, self.ctx = cache.pages.cuda(), cache.table.cuda(), torch.tensor(ctx, dtype=I32, device="cuda")
        self.cos, self.sin = (x.cuda() for x in layer_ref.tables(max(ctx) + self.max_t, D))
        # q, k and v of the recurrence and the cache, and the wide attention's queries: a convolution each
        self.channels = [H * D, H * D, H * D, WIDE * D]
        self.windows = [r(n, KW - 1, c).to(BF16).cuda() for c in self.channels]
        self.weights = [(0.5 * r(c, KW)).cuda() for c in self.channels]
        self.slots = torch.randperm(n, generator=g).to(I32).cuda()
        self.x = [[r(total, c).to(BF16).cuda() for c in self.channels] for _ in range(steps)]
        self.a, self.b = [r(total, H, D).cuda() for _ in range(steps)], [r(total, H).cuda() for _ in range(steps)]
        self.tokens = [torch.randint(0, WIDE * D, (total,), generator=g).to(I32).cuda() for _ in range(steps)]
        self.u, self.u_last = [torch.rand(total, generator=g).cuda() for _ in range(steps)], torch.rand(n, generator=g).cuda()
        # (a run's own memory, filled with what no call may leave behind)
        self.ws = torch.zeros(kda.KDA_KV4_TREE_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
        self.pool, self.pages = self.pool0.clone(), self.pages0.clone()
        self.node, self.status = torch.ones(n, dtype=I32, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
        f = lambda *s, dtype=BF16: torch.full(s, float("nan"), dtype=dtype, device="cuda")  # noqa: E731
        i = lambda *s: torch.full(s, 99, dtype=I32, device="cuda")  # noqa: E731
        self.out = [dict(y=[f(total, c) for c in self.channels], o=f(total, H, D, dtype=F32), narrow=f(total, H, D),
                         wide=[f(total, WIDE, D) for _ in range(2)], again=f(total, H, D), accepted=i(n), path=i(n, self.max_t), token=i(n))
                    for _ in range(steps)]

    def reset(self):
        self.pool.copy_(self.pool0)
        self.pages.copy_(self.pages0)
        self.node.fill_(1)
        self.status.zero_()
        for o in self.out:
            for t in (*o["y"], o["o"], o["narrow"], *o["wide"], o["again"]):
                t.fill_(float("nan"))
            for name in ("accepted", "path", "token"):
                o[name].fill_(99)

    def run(self, flags, stream=None):
        kw = dict(cu_seqlens=self.cu, max_t=self.max_t, flags=flags, stream=stream)
        L, view = self.lib, lambda t, h: t.view(self.total, h, D)  # noqa: E731
        for s, o in enumerate(self.out):
            for w, x, weight, y in zip(self.windows, self.x[s], self.weights, o["y"]):
                L.kda_conv_step_tree(w, self.slots, x, weight, self.tree, y, self.status, **kw)
            q, k, v, wide = (view(y, c // D) for y, c in zip(o["y"], self.channels))
            L.kda_step_tree(self.pool, self.table, q, k, v, self.a[s], self.b[s], self.tree, o["o"], self.status, accepted=self.node, **kw)
            L.kda_kv4_append_tree(self.pages, self.ptab, self.ctx, k, v, self.tree, self.status, cos=self.cos, sin=self.sin, **kw)
            for q, to in ((wide, o["wide"][0]), (o["wide"][0], o["wide"][1]), (q, o["narrow"]), (o["narrow"], o["again"])):
                L.kda_kv4_attend_tree(self.pages, self.ptab, self.ctx, q, self.tree, to, self.ws, self.status, cos=self.cos, sin=self.sin, **kw)
            L.kda_accept(o["wide"][1].view(self.total, -1), self.tokens[s], self.u[s], self.u_last, o["accepted"], self.node, o["path"], o["token"],
                         self.status, q=o["wide"][0].view(self.total, -1), tree=self.tree, **kw)

    def results(self):
        torch.cuda.synchronize()
        assert self.status.item() == 0 and not self.ws[:2048].any()
        every = [t for o in self.out for t in (*o["y"], o["o"], o["narrow"], *o["wide"], o["again"], o["accepted"], o["path"], o["token"])]
        return [t.clone() for t in (*every, self.pool, self.pages, self.node)]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


CASES = [(F32, [(9, "wide"), (5, "chain"), (1, "chain"), (7, "star")], [0, 33, 100, 17], 6),
         (F16, [(1 + (7 * i) % 23, ("wide", "star", "forest")[i % 3]) for i in range(24)], [(61 * i) % 700 for i in range(24)], 4),
         (F16, [(12, "wide")], [5000], 4)]


@pytest.mark.parametrize("pool_dtype,shapes,ctx,steps", CASES)
def test_dependent_launches(libs, pool_dtype, shapes, ctx, steps):
    c = Chain(libs[pool_dtype], pool_dtype, shapes, ctx, steps)
    c.run(0)
    want = c.results()
    assert not any(t.isnan().any() for t in want[:-2] if t.is_floating_point())
    assert max(int(o["accepted"].max()) for o in c.out) > 1 or c.n == 1     # the steps go on from more than their roots
    for _ in range(5):
        c.reset()
        torch.cuda.synchronize()
        c.run(kda.KDA_LAUNCH_PDL)
        assert same(c.results(), want)
    # a graph of the whole chain, replayed
    graph = torch.cuda.CUDAGraph()
    c.reset()
    with torch.cuda.graph(graph):
        c.run(kda.KDA_LAUNCH_PDL)
    for _ in range(3):
        c.reset()
        graph.replay()
        assert same(c.results(), want)
    # and behind itself: a replay whose first calls meet the last ones of the one before
    c.reset()
    graph.replay()
    c.node.fill_(1)
    c.pool.copy_(c.pool0)
    graph.replay()
    assert same(c.results(), want)


@pytest.mark.parametrize("flags", [0, kda.KDA_LAUNCH_PDL])
@pytest.mark.parametrize("how", ["argument", "current"])
def test_another_stream(libs, how, flags):
    """Inputs that come late on a stream: a call that went to another one would read the NaN before them."""
    c = Chain(libs[F32], F32, *CASES[0][1:3], 2, seed=4)
    c.run(0)
    want = c.results()
    late = [(t, t.clone()) for s in range(2) for t in (*c.x[s], c.a[s], c.b[s], c.u[s])]
    c.reset()
    for t, _ in late:
        t.fill_(float("nan"))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        for t, value in late:
            t.copy_(value)
        if how == "current":
            c.run(flags)
    if how == "argument":
        c.run(flags, stream=side)
    assert same(c.results(), want)


def test_two_streams_at_a_time(libs):
    """Two chains, each on a stream and a workspace of its own, share the GPU (and an SM's tensor memory)."""
    chains = [Chain(libs[F16], F16, [(24, "wide")] * 3, [900, 1500, 333], 6, seed=5 + i) for i in range(2)]
    want = []
    for c in chains:
        c.run(0)
        want.append(c.results())
        c.reset()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in chains]
    for flags in (0, kda.KDA_LAUNCH_PDL):
        for c, s in zip(chains, streams):
            with torch.cuda.stream(s):
                torch.cuda._sleep(2_000_000)
                c.run(flags)
        for c, w in zip(chains, want):
            assert same(c.results(), w)
            c.reset()
        torch.cuda.synchronize()


def test_a_chain_has_the_bits_of_kda_kv4_attend(libs):
    """Up to 48 query rows a head: the same keys in the same order, masked or not."""
    lib, g = libs[F32], torch.Generator().manual_seed(2)
    ws = torch.zeros(kda.KDA_KV4_TREE_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")  # noqa: E731
    for ctx, lens in (([200, 31, 64], [7, 1, 8]), ([5000], [4]), ([0, 1, 17, 333], [3, 2, 1, 8])):
        cu = [0]
        for t in lens:
            cu.append(cu[-1] + t)
        tree = ref.masks([ref.parents(t, "chain") for t in lens])
        for dim in (64, 128):
            cache = layer_ref.Cache([c + t for c, t in zip(ctx, lens)], 2, dim, 64, g)
            cos, sin = (x.cuda() for x in layer_ref.tables(max(ctx) + 8, dim))
            for dtype in (F32, F16, BF16):
                for grp, window in ((1, 0), (4, 0), (4, 40)):
                    q = torch.randn(sum(lens), 2 * grp, dim, generator=g).to(dtype).cuda()
                    o, o2, st = torch.zeros_like(q), torch.ones_like(q), i32([0])
                    kw = dict(cu_seqlens=i32(cu), max_t=8, cos=cos, sin=sin, window=window)
                    common = (cache.pages.cuda(), cache.table.cuda(), i32(ctx), q)
                    lib.kda_kv4_attend(*common, o, ws, st, **kw)
                    lib.kda_kv4_attend_tree(*common, tree, o2, ws, st, **kw)
                    assert st.item() == 0 and torch.equal(o, o2)
