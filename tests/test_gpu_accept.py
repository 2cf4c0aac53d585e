"""kda_accept against the walk in 64 bits: every output is a whole number and has to be equal."""
import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

import _tree_ref as ref

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32


@pytest.fixture(scope="module")
def lib(built_libs):
    return kda.KdaLibrary(F32)


def ints(v, dtype=I32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def inputs(pars, vocab, dtype, drawn, seed=0, near=0.7, peak=3.0):
    """p, q, tokens, u, u_last on the CPU: drafts near the target, drawn from q or q's best."""
    g = torch.Generator().manual_seed(seed)
    total = sum(map(len, pars))
    logits = peak * torch.randn(total, vocab, generator=g)
    draft = logits + near * torch.randn(total, vocab, generator=g)
    p, q = torch.softmax(logits, -1).to(dtype), torch.softmax(draft, -1).to(dtype)
    tokens, at = torch.zeros(total, dtype=I32), 0
    for par in pars:
        used = {}
        for i, up in enumerate(par):
            if up >= 0:
                if drawn:
                    tokens[at + i] = int(torch.multinomial(q[at + up].float(), 1, generator=g))
                else:
                    best = torch.topk(draft[at + up], min(vocab, 8)).indices
                    tokens[at + i] = int(best[used.get(up, 0) % len(best)])
                    used[up] = used.get(up, 0) + 1
        at += len(par)
    return p, q if drawn else None, tokens, torch.rand(total, generator=g), torch.rand(len(pars), generator=g)


def run(lib, pars, p, q, tokens, u, u_last, tree=True, equal=False, max_t=None, cu=None, tree_t=None, stream=None):
    n, lens = len(pars), [len(x) for x in pars]
    max_t = max(lens) if max_t is None else max_t
    if cu is None:
        cu = [0]
        for t in lens:
            cu.append(cu[-1] + t)
    out = [torch.full(s, 99, dtype=I32, device="cuda") for s in ((n,), (n,), (n, max_t), (n,))]
    st = ints([0])
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    lib.kda_accept(c(p), c(tokens), c(u), c(u_last), *out, st, q=c(q), tree=(ref.masks(pars) if tree_t is None else tree_t) if tree else None,
                   cu_seqlens=None if equal else ints(cu), max_t=max_t, stream=stream)
    torch.cuda.synchronize()
    return [x.cpu() for x in out], st.item()


def check(pars, p, q, tokens, u, u_last, out):
    accepted, node, path, token = out
    at = 0
    for r, par in enumerate(pars):
        t = len(par)
        if t == 0:
            assert (accepted[r], node[r], token[r]) == (0, 0, -1) and (path[r] == -1).all()
            continue
        sl = slice(at, at + t)
        want, nxt = ref.accept(p[sl], None if q is None else q[sl], tokens[sl], par, u[sl], u_last[r])
        assert path[r].tolist() == [at + i for i in want] + [-1] * (path.shape[1] - len(want)), r
        assert accepted[r] == len(want) and node[r] == want[-1] + 1, r
        assert token[r] == nxt, (r, int(token[r]), nxt)
        at += t


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("shapes,vocab,near", [
    ([(5, "chain")], 32000, 0.5),
    ([(8, "chain")] * 9, 1000, 0.2),
    ([(64, "wide")] * 3, 777, 1.0),
    ([(33, "star"), (0, "chain"), (1, "chain"), (17, "wide"), (20, "forest")], 4099, 2.0),
    ([(6, "wide")] * 40, 37, 0.5),
    ([(3, "star")], 1, 0.5),
    ([(9, "star")] * 5, 2, 3.0),
])
def test_accept_against_fp64(lib, dtype, drawn, shapes, vocab, near):
    pars = [ref.parents(t, k, i) for i, (t, k) in enumerate(shapes)]
    x = inputs(pars, vocab, dtype, drawn, seed=vocab + len(pars), near=near)
    out, st = run(lib, pars, *x)
    assert st == 0
    check(pars, *x, out)


def test_accept_chains_without_masks(lib):
    pars = [ref.parents(8, "chain")] * 7
    x = inputs(pars, 5003, F32, True, near=0.3)
    a, st = run(lib, pars, *x, tree=False, equal=True)
    assert st == 0
    check(pars, *x, a)
    b, _ = run(lib, pars, *x)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("drawn", [True, False])
def test_accept_rows_apart_and_off_their_alignment(lib, drawn):
    """Rows of any alignment, p's and q's alike and not."""
    pars = [ref.parents(12, "star", 1), ref.parents(9, "wide", 2)]
    for dtype in (F32, BF16):
        p, q, *rest = inputs(pars, 1237, dtype, drawn, near=1.5)
        for (a, sa), (b, sb) in (((1, 1240), (1, 1240)), ((3, 1241), (0, 1243)), ((0, 1248), (5, 1237))):
            rows = []
            for t, off, stride in ((p, a, sa), (q, b, sb)):
                if t is None:
                    rows.append(None)
                    continue
                hold = torch.full((off + t.shape[0] * stride,), float("nan"), dtype=dtype, device="cuda")
                view = hold[off:].view(-1, stride)[:, :1237] if stride >= 1237 else None
                view.copy_(t)
                rows.append(view)
            out, st = run(lib, pars, *rows, *rest)
            assert st == 0
            check(pars, p, q, *rest, out)


def test_accept_ties_zeros_and_ones(lib):
    """Sums that are exact in any order, and random numbers on their borders."""
    vocab = 300
    p = torch.zeros(8, vocab)
    p[:, 10], p[:, 20], p[:, 250] = 0.5, 0.25, 0.25
    par1 = [[-1]] * 8
    last = torch.tensor([0.0, 0.49999997, 0.5, 0.74999994, 0.75, 0.99999994, 1.0, float("nan")])
    out, st = run(lib, par1, p, None, torch.zeros(8, dtype=I32), torch.zeros(8), last)
    # the sum has to pass u_last: on a border the next one; past the end, or not a number, the last
    assert st == 0 and out[3].tolist() == [10, 10, 20, 20, 250, 250, 250, 250]
    # u q(x) = p(x) rejects, just below accepts; p = q accepts for every u below 1
    par2 = [[-1, 0]] * 4
    p2, q2 = p.repeat_interleave(1, 0)[:8].clone(), p.clone()
    q2[:, 10], q2[:, 20], q2[:, 250] = 1.0, 0.0, 0.0
    tokens = torch.tensor([0, 10] * 4, dtype=I32)
    u = torch.tensor([0, 0.5, 0, 0.49999997, 0, 0.0, 0, 1.0])
    x = (p2, q2, tokens, u, torch.tensor([0.0, 0.6, 0.0, 0.5]))
    out, st = run(lib, par2, *x)
    assert st == 0 and out[0].tolist() == [1, 2, 2, 1] and out[3].tolist() == [20, 20, 10, 250]
    check(par2, *x, out)
    x = (p2, p2, tokens, torch.full((8,), 0.99999994), torch.tensor([0.0, 0.6, 0.0, 0.5]))
    out, st = run(lib, par2, *x)
    assert st == 0 and out[0].tolist() == [2] * 4
    check(par2, *x, out)


def test_accept_nothing_left_falls_back_to_the_targets_row(lib):
    """p below q everywhere (a row that lost mass to rounding): W is zero after the rejection."""
    p = torch.zeros(2, 50)
    p[0, 3], p[0, 4] = 0.25, 0.5
    q = torch.zeros(2, 50)
    q[0, 3], q[0, 4] = 0.4, 0.6
    x = (p, q, torch.tensor([0, 3], dtype=I32), torch.tensor([0.0, 0.9]), torch.tensor([0.5]))
    out, st = run(lib, [[-1, 0]], *x)
    assert st == 0 and out[0].tolist() == [1] and out[3].tolist() == [4]
    check([[-1, 0]], *x, out)
    # given drafts that hold all of the mass
    p = torch.zeros(3, 50)
    p[0, 7], p[0, 9] = 0.75, 0.125
    x = (p, None, torch.tensor([0, 7, 9], dtype=I32), torch.tensor([0.0, 0.8, 0.9]), torch.tensor([0.9]))
    out, st = run(lib, [[-1, 0, 0]], *x)
    assert st == 0 and out[3].tolist() == [9]
    check([[-1, 0, 0]], *x, out)


def test_accept_the_same_draft_twice(lib):
    for drawn in (True, False):
        pars = [[-1, 0, 0, 0, 0]] * 30
        p, q, tokens, u, last = inputs(pars, 211, F32, drawn, near=2.5, seed=3)
        tokens[:] = tokens.view(30, 5)[:, 1:2].expand(30, 5).reshape(-1)
        out, st = run(lib, pars, p, q, tokens, u, last)
        assert st == 0
        check(pars, p, q, tokens, u, last, out)


def test_accept_bad_values_ids_and_offsets(lib):
    pars = [[-1, 0, 1, 0]] * 4
    p, q, tokens, u, last = inputs(pars, 97, F32, True, near=0.1)
    nan, inf = float("nan"), float("inf")
    # NaN and negative entries count as zero
    p2, q2 = p.clone(), q.clone()
    p2[0, 5:40], q2[0, 50:60], p2[4, 60:], q2[5] = nan, -1.0, -inf, nan
    out, st = run(lib, pars, p2, q2, tokens, u, last)
    assert st == 0
    check(pars, p2, q2, tokens, u, last, out)
    # a row without weight, or with an infinite one, where the next token is drawn
    for row in (torch.zeros(97), torch.full((97,), nan), p[0].clone().index_fill_(0, torch.tensor([3]), inf)):
        p2 = p.clone()
        p2[0] = row
        t2 = tokens.clone()
        t2[1:4] = 90
        if row[90] > 0:
            u2 = torch.full_like(u, 1.0)
        else:
            u2 = u
        out, st = run(lib, pars, p2, None, t2, u2, last)
        assert st == kda.KDA_ERR_ARG and out[3][0] == -1 and out[0][0] == 1 and out[1][0] == 1 and out[2][0].tolist() == [0, -1, -1, -1]
        check(pars[1:], p2[4:], None, t2[4:], u2[4:], last[1:], [x[1:] if x.dim() == 1 else torch.where(x[1:] >= 0, x[1:] - 4, x[1:]) for x in out])
    # ids outside the vocabulary: not tested, what hangs on them not reached
    t2 = tokens.clone()
    t2[1], t2[7], t2[9] = 97, -1, 2 ** 31 - 1
    out, st = run(lib, pars, p, q, t2, u, last)
    assert st == kda.KDA_ERR_ARG
    check(pars, p, q, t2, u, last, out)
    # token offsets
    for cu, bad in (([0, 4, 3, 12, 16], {1, 2}), ([0, 4, 8, 13, 16], {2}), ([-1, 3, 8, 12, 16], {0, 1}), ([0, 4, 8, 13, 17], {2, 3})):
        out, st = run(lib, pars, p, q, tokens, u, last, cu=cu)
        assert st == kda.KDA_ERR_ARG
        for r in bad:
            assert (out[0][r], out[1][r], out[3][r]) == (0, 0, -1) and (out[2][r] == -1).all()


def test_accept_no_tokens_at_all(lib):
    e = torch.zeros(0, 12)
    out, st = run(lib, [[], []], e, None, torch.zeros(0, dtype=I32), torch.zeros(0), torch.rand(2), max_t=3, cu=[0, 0, 0])
    assert st == 0 and out[0].tolist() == [0, 0] and out[3].tolist() == [-1, -1] and (out[2] == -1).all()


def test_accept_on_another_stream_and_captured(lib):
    pars = [ref.parents(7, "wide", i) for i in range(5)]
    x = inputs(pars, 2001, BF16, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, st = run(lib, pars, *x, stream=side)
    assert st == 0
    check(pars, *x, out)
    p, q, tokens, u, last = (t.cuda() for t in x)
    cu, tree, status = ints([0, 7, 14, 21, 28, 35]), ref.masks(pars), ints([0])
    outs = [torch.zeros(s, dtype=I32, device="cuda") for s in ((5,), (5,), (5, 7), (5,))]
    call = lambda: lib.kda_accept(p, tokens, u, last, *outs, status, q=q, tree=tree, cu_seqlens=cu, max_t=7)  # noqa: E731
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    y = inputs(pars, 2001, BF16, True, seed=8)
    for dst, src in zip((p, q, tokens, u, last), y):
        dst.copy_(src)
    graph.replay()
    torch.cuda.synchronize()
    check(pars, *y, [t.cpu() for t in outs])
