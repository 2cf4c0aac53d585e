"""The calls of a step over trees of drafted tokens together, as a hybrid stack makes them: convolution, recurrence and
attention over the trees, acceptance, and the accepted paths kept; against the same tokens one chain at a time through
the calls without trees."""
import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

import _layer_ref as layer_ref
import _tree_ref as ref

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32
HV, K, V, KW = 2, 64, 32, 4                # the KDA layer
HQ, HKV, DIM, PAGE = 4, 2, 64, 16          # the attention layer
VOCAB, N, T = 61, 4, 9
C = 2 * HV * K + HV * V


class Stack:
    """The memory of one KDA layer and one attention layer; `cols` snapshot columns a request."""

    def __init__(self, lib, pool_dtype, cols, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.lib, self.cols = lib, cols
        self.pool = (0.3 * torch.randn(N * cols, HV, K, V, generator=g)).to(pool_dtype).cuda()
        self.table = torch.arange(N * cols, dtype=I32, device="cuda").view(N, cols)
        self.node = torch.ones(N, dtype=I32, device="cuda")
        # the first column of every request is the state to start from
        self.start = self.pool[self.table[:, 0].long()].clone()
        self.window = torch.randn(N + 1, KW - 1, C, generator=g).to(BF16).cuda()
        self.conv_slot = torch.tensor([2, 0, 4, 1, -1], dtype=I32, device="cuda")      # the last one: rows of no request
        self.weight = (0.5 * torch.randn(C, KW, generator=g)).cuda()
        pages = 8
        self.pages = torch.zeros((N + 1) * pages, HKV, PAGE // 16, 18 * DIM, dtype=torch.uint8, device="cuda")
        self.ptab = torch.randperm((N + 1) * pages, generator=g).to(I32).cuda().view(N + 1, pages)
        self.ctx = torch.zeros(N + 1, dtype=I32, device="cuda")
        self.cos, self.sin = (x.cuda() for x in layer_ref.tables(pages * PAGE, DIM))
        self.ws = torch.zeros(kda.KDA_KV4_TREE_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(1, dtype=I32, device="cuda")


def inputs(seed, total):
    """One step's inputs of every token: the convolution's and the gates', the attention's, the target's and the drafts' probabilities."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    logits = 2 * r(total, VOCAB)
    draft = logits + 0.5 * r(total, VOCAB)
    return {"x": r(total, C).to(BF16).cuda(), "a": r(total, HV, K).cuda(), "b": r(total, HV).cuda(),
            "q": r(total, HQ, DIM).to(BF16).cuda(), "k": r(total, HKV, DIM).to(BF16).cuda(), "v": r(total, HKV, DIM).to(BF16).cuda(),
            "p": torch.softmax(logits, -1).cuda(), "d": torch.softmax(draft, -1).cuda(),
            "u": torch.rand(total, generator=g).cuda(), "u_last": torch.rand(N, generator=g).cuda()}


def split(y):
    rows = y.shape[0]
    return (y[:, :HV * K].reshape(rows, HV, K).contiguous(), y[:, HV * K:2 * HV * K].reshape(rows, HV, K).contiguous(),
            y[:, 2 * HV * K:].reshape(rows, HV, V).contiguous())


def tree_step(s, i, tree, tokens, cu, cu_pad):
    """A step over the trees, and the accepted paths kept.  No shape depends on what is accepted: rows that no path fills
    go to a last request that is padding."""
    L, total = s.lib, i["x"].shape[0]
    new = lambda *shape, dtype=F32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    y, o_kda, o_att = new(total, C, dtype=BF16), new(total, HV, V), new(total, HQ, DIM, dtype=BF16)
    L.kda_conv_step_tree(s.window, s.conv_slot[:N], i["x"], s.weight, tree, y, s.status, cu_seqlens=cu, max_t=T)
    q, k, v = split(y)
    L.kda_step_tree(s.pool, s.table, q, k, v, i["a"], i["b"], tree, o_kda, s.status, cu_seqlens=cu, max_t=T, accepted=s.node)
    L.kda_kv4_append_tree(s.pages, s.ptab[:N], s.ctx[:N], i["k"], i["v"], tree, s.status, cu_seqlens=cu, max_t=T, cos=s.cos, sin=s.sin)
    L.kda_kv4_attend_tree(s.pages, s.ptab[:N], s.ctx[:N], i["q"], tree, o_att, s.ws, s.status, cu_seqlens=cu, max_t=T, cos=s.cos, sin=s.sin)
    accepted, token = new(N, dtype=I32), new(N, dtype=I32)
    path = new(N, T, dtype=I32)
    L.kda_accept(i["p"], tokens, i["u"], i["u_last"], accepted, s.node, path, token, s.status, q=i["d"], tree=tree, cu_seqlens=cu, max_t=T)
    # the paths' rows first, then rows of no request, in a batch of `total` rows
    flat = path.view(-1)
    order = torch.argsort((flat < 0).int(), stable=True)[:total]
    rows = flat[order].clamp(min=0).long()
    cu_pad[1:N + 1] = accepted.cumsum(0).int()
    cu_pad[N + 1:].fill_(total)
    s.ctx[N:].fill_(-total)
    yk = new(total, C, dtype=BF16)
    L.kda_conv_step(s.window, s.conv_slot, i["x"][rows], s.weight, yk, s.status, cu_seqlens=cu_pad, max_t=total)
    L.kda_kv4_append(s.pages, s.ptab, s.ctx, i["k"][rows], i["v"][rows], s.status, cu_seqlens=cu_pad, max_t=total, cos=s.cos, sin=s.sin)
    s.ctx[:N] += accepted
    return o_kda, o_att, accepted, path, token


def make_trees(step):
    pars = [ref.parents(T if r else 3, ("wide", "star", "chain", "wide")[r], 10 * step + r) for r in range(N)]
    cu = [0]
    for p in pars:
        cu.append(cu[-1] + len(p))
    g = torch.Generator().manual_seed(100 + step)
    return pars, torch.tensor(cu, dtype=I32, device="cuda"), torch.randint(0, VOCAB, (cu[-1],), generator=g)


def draft_tokens(pars, d, seed):
    """Each token drawn from its parent's draft distribution."""
    g = torch.Generator().manual_seed(seed)
    out, at = [], 0
    for par in pars:
        for up in par:
            out.append(0 if up < 0 else int(torch.multinomial(d[at + up].cpu(), 1, generator=g)))
        at += len(par)
    return torch.tensor(out, dtype=I32, device="cuda")


@pytest.mark.parametrize("pool_dtype", [F32, F16])
def test_steps_over_trees_are_the_steps_of_their_paths(built_libs, pool_dtype):
    lib = kda.KdaLibrary(pool_dtype)
    s = Stack(lib, pool_dtype, T)
    c = Stack(lib, pool_dtype, T)       # one chain of accepted tokens, by the calls without trees
    cu_pad = torch.zeros(N + 2, dtype=I32, device="cuda")
    for step in range(4):
        pars, cu, _ = make_trees(step)
        total = int(cu[-1])
        i = inputs(step, total)
        tokens = draft_tokens(pars, i["d"], step)
        o_kda, o_att, accepted, path, token = tree_step(s, i, ref.masks(pars), tokens, cu, cu_pad)
        assert s.status.item() == 0
        at = 0
        for r, par in enumerate(pars):
            sl = slice(at, at + len(par))
            want, nxt = ref.accept(i["p"][sl].cpu(), i["d"][sl].cpu(), tokens[sl].cpu(), par, i["u"][sl].cpu(), i["u_last"][r].cpu())
            assert path[r].tolist()[:len(want)] == [at + j for j in want] and accepted[r].item() == len(want) and token[r].item() == nxt
            at += len(par)
        # the same tokens as chains
        lens = accepted.tolist()
        rows = torch.cat([path[r, :lens[r]] for r in range(N)]).long()
        cu2 = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=I32, device="cuda")
        pick = {n: i[n][rows].contiguous() for n in ("x", "a", "b", "q", "k", "v")}
        y = torch.empty(len(rows), C, dtype=BF16, device="cuda")
        lib.kda_conv_step(c.window, c.conv_slot[:N], pick["x"], c.weight, y, c.status, cu_seqlens=cu2, max_t=T)
        q, k, v = split(y)
        oc = torch.empty(len(rows), HV, V, device="cuda")
        lib.kda_step(c.pool, c.table, q, k, v, pick["a"], pick["b"], oc, c.status, cu_seqlens=cu2, max_t=T, accepted=c.node)
        lib.kda_kv4_append(c.pages, c.ptab[:N], c.ctx[:N], pick["k"], pick["v"], c.status, cu_seqlens=cu2, max_t=T, cos=c.cos, sin=c.sin)
        oa = torch.empty(len(rows), HQ, DIM, dtype=BF16, device="cuda")
        lib.kda_kv4_attend(c.pages, c.ptab[:N], c.ctx[:N], pick["q"], oa, c.ws, c.status, cu_seqlens=cu2, max_t=T, cos=c.cos, sin=c.sin)
        c.ctx[:N] += accepted
        c.node = accepted.clone()
        assert c.status.item() == 0 and torch.equal(c.ctx[:N], s.ctx[:N])
        # the recurrence: fp32 roundings of four steps of up to nine tokens; an fp16 pool may round a state's last bit differently
        # (2^-11 of states up to 4), which an output of 64 products of unit vectors then carries
        lim = 1e-5 if pool_dtype == F32 else 2e-3
        assert (o_kda[rows] - oc).abs().max() <= lim
        for r in range(N):
            a, b = s.pool[s.table[r, s.node[r] - 1].item()].float(), c.pool[c.table[r, lens[r] - 1].item()].float()
            assert (a - b).abs().max() <= (2e-5 if pool_dtype == F32 else 8e-3)
        # windows and cached tokens bit for bit: a token's bytes of every page
        assert torch.equal(s.window, c.window)
        same_cache(s, c)
        # attention: bf16 outputs of values up to about 4, each call within its rounding and 2^-9 of them (probabilities in 11 bits)
        assert (o_att[rows].float() - oa.float()).abs().max() <= 4 * (2 * 2.0 ** -8 + 2 * 2.0 ** -9)


def same_cache(s, c):
    """The tokens before ctx_len, byte for byte (behind it a tree leaves its own)."""
    for r in range(N):
        for p in range(int(s.ctx[r])):
            for st in ((s, c),):
                a, b = (x.pages[x.ptab[r, p // PAGE].item(), :, p % PAGE // 16] for x in st)
                w = p % 16
                assert torch.equal(a[:, w * DIM // 2:(w + 1) * DIM // 2], b[:, w * DIM // 2:(w + 1) * DIM // 2])
                assert torch.equal(a[:, 16 * DIM + w * DIM // 16:16 * DIM + (w + 1) * DIM // 16], b[:, 16 * DIM + w * DIM // 16:16 * DIM + (w + 1) * DIM // 16])


def test_a_step_over_trees_captured_and_replayed(built_libs):
    """A whole step as one graph, replayed on other inputs, against the eager calls."""
    lib = kda.KdaLibrary(F32)
    pars, cu, _ = make_trees(0)
    total, tree = int(cu[-1]), ref.masks(pars)
    i = inputs(0, total)
    tokens = draft_tokens(pars, i["d"], 0)
    eager, graphed = Stack(lib, F32, T), Stack(lib, F32, T)
    pad = [torch.zeros(N + 2, dtype=I32, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):       # a warm-up on memory of its own
        tree_step(Stack(lib, F32, T), i, tree, tokens, cu, torch.zeros(N + 2, dtype=I32, device="cuda"))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tree_step(graphed, i, tree, tokens, cu, pad[1])
    for step in range(3):
        fresh = inputs(20 + step, total)
        for name in i:
            i[name].copy_(fresh[name])
        tokens.copy_(draft_tokens(pars, i["d"], step))
        want = tree_step(eager, i, tree, tokens, cu, pad[0])
        graph.replay()
        torch.cuda.synchronize()
        assert eager.status.item() == 0 and graphed.status.item() == 0
        for a, b in zip(want, out):
            assert torch.equal(a, b)
        assert torch.equal(eager.pool, graphed.pool) and torch.equal(eager.pages, graphed.pages) and torch.equal(eager.window, graphed.window)
