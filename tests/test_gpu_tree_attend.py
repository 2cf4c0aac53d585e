"""kda_kv4_append_tree and kda_kv4_attend_tree: bytes bit for bit, and attention against fp64 with the tolerance derived in _layer_ref."""
import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

import _layer_ref as ref
import _tree_ref as tree_ref
from test_gpu_kv4 import append_reference, ragged

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def lib(built_libs):
    return kda.KdaLibrary(F32)


@pytest.fixture(scope="module")
def workspace():
    return torch.zeros(kda.KDA_KV4_TREE_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def depths(pars):
    return [len(p) - 1 for par in pars for p in tree_ref.ancestors(par)]


@pytest.mark.parametrize("heads,dim,page,ctx,shapes,dtype,rot,inter", [
    (2, 128, 64, [0, 60, 127], ["wide", "chain", "star"], BF16, 128, False),
    (3, 64, 16, [7, 0, -20], ["forest", "wide", "wide"], F16, 32, True),
    (1, 128, 32, [100], ["wide"], F32, 64, False),
    (2, 64, 48, [5], ["wide"], BF16, 0, False),
])
def test_append_tree_is_bit_exact(lib, heads, dim, page, ctx, shapes, dtype, rot, inter):
    g = torch.Generator().manual_seed(heads * dim)
    pars = [tree_ref.parents(20 if i != 1 else 3, s, i) for i, s in enumerate(shapes)]
    lens = [len(p) for p in pars]
    total = sum(lens)
    cache = ref.Cache([max(0, c + t) for c, t in zip(ctx, lens)], heads, dim, page, g)
    rows = max(c + t for c, t in zip(ctx, lens))
    cos, sin = ref.tables(rows, rot) if rot else (None, None)
    x = (torch.randn(2, total, heads, dim, generator=g) * 3).to(dtype)
    od = BF16 if dtype == F32 else dtype
    pages, st = cache.pages.cuda(), i32([0])
    ko, vo = (torch.full((total, heads, dim), float("nan"), dtype=od, device="cuda") for _ in range(2))
    lib.kda_kv4_append_tree(pages, cache.table.cuda(), i32(ctx), x[0].cuda(), x[1].cuda(), tree_ref.masks(pars), st, cu_seqlens=ragged(lens),
                            max_t=max(lens), cos=None if cos is None else cos.cuda(), sin=None if sin is None else sin.cuda(),
                            interleaved=inter, k_out=ko, v_out=vo)
    torch.cuda.synchronize()
    assert st.item() == 0
    # keys rotated beforehand by their depth, then stored as they are
    k = x[0].float()
    if rot:
        pos = torch.tensor([max(0, ctx[r] + d) for r, par in enumerate(pars) for d in depths([par])])
        k = ref.rotate32(k, cos[pos], sin[pos], inter)
    want, (kv, vv) = append_reference(cache.pages, cache.table, page, ctx, lens, k, x[1], None, None, False)
    assert torch.equal(pages.cpu(), want)
    assert torch.equal(ko.cpu().double(), kv) and torch.equal(vo.cpu().double(), vv)


def run(lib, ws, heads, grp, dim, page, ctx, pars, dtype, rot, inter, window=0, seed=0, ks=1.0, vs=1.0, scale=None, q_gain=1.5, poison=None,
        edit=None, equal=False, cache=None, stream=None):
    g = torch.Generator().manual_seed(seed)
    lens = [len(p) for p in pars]
    total, hq = sum(lens), heads * grp
    ends = [c + t if c >= 0 else 0 for c, t in zip(ctx, lens)]
    if cache is None:
        cache = ref.Cache(ends, heads, dim, page, g, poison=poison)
    cos, sin = ref.tables(max(1, max(ends)), rot) if rot else (None, None)
    q = (torch.randn(total, hq, dim, generator=g) * q_gain).to(dtype)
    if edit is not None:
        edit(q)
    o = torch.full((total, hq, dim), float("nan"), dtype=dtype, device="cuda")
    st = i32([0])
    args = [cache.pages.cuda(), cache.table.cuda(), i32(ctx), q.cuda(), tree_ref.masks(pars), o, ws, st]
    torch.cuda.synchronize()
    lib.kda_kv4_attend_tree(*args, cu_seqlens=None if equal else ragged(lens), max_t=max(lens), cos=None if cos is None else cos.cuda(),
                            sin=None if sin is None else sin.cuda(), interleaved=inter, window=window, scale=scale, k_scale=ks, v_scale=vs,
                            stream=stream)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert not ws[:2048].any(), "the workspace's counters are not back at zero"
    want, err, big, top = tree_ref.attend(cache, ctx, pars, q, cos, sin, inter, window, scale, ks, vs)
    got = o.cpu().double()
    lim = ref.attend_tolerance(want, err, big, top, dtype, dtype != BF16)
    assert torch.equal(got.isnan(), want.isnan())
    bad = (got - want).abs() > lim
    assert not bad.any(), f"worst {((got - want).abs() / lim).nan_to_num(0).max():.3g} of the bound"
    return got, want


def trees(*shapes):
    return [tree_ref.parents(t, k, i) for i, (t, k) in enumerate(shapes)]


@pytest.mark.parametrize("heads,grp,dim,page,ctx,shapes,dtype,rot,inter,window", [
    (1, 1, 128, 16, [0], [(1, "chain")], BF16, 0, False, 0),                      # a single key
    (2, 4, 128, 64, [15, 16, 300], [(7, "wide"), (8, "star"), (2, "chain")], BF16, 128, False, 0),
    (2, 6, 64, 16, [37, 0, 130], [(12, "forest"), (64, "wide"), (1, "chain")], F16, 64, True, 0),
    (1, 8, 128, 128, [1000], [(9, "wide")], F32, 64, False, 0),
    (3, 5, 128, 48, [50, -12, 5, 9], [(33, "wide"), (12, "wide"), (3, "star"), (0, "chain")], BF16, 128, False, 0),
    (2, 2, 128, 16, [400, 33], [(14, "wide"), (14, "chain")], F16, 128, False, 1),          # only itself
    (1, 16, 128, 64, [700, 20], [(30, "wide"), (30, "chain")], BF16, 128, True, 100),
    (1, 33, 64, 16, [257], [(20, "chain")], BF16, 64, False, 7),                            # shorter than the paths
    (2, 8, 128, 128, [500, 31], [(64, "wide"), (63, "chain")], BF16, 128, False, 0),
    (1, 4, 128, 32, [96, 95, 97], [(40, "forest")] * 3, BF16, 128, False, 33),
    (1, 2, 64, 16, [0, 0], [(64, "forest"), (31, "forest")], F32, 64, True, 0),              # no context
])
def test_attend_tree_against_fp64(lib, workspace, heads, grp, dim, page, ctx, shapes, dtype, rot, inter, window):
    run(lib, workspace, heads, grp, dim, page, ctx, trees(*shapes), dtype, rot, inter, window, seed=heads * grp + dim)


@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, F32)])
def test_attend_tree_long_context_over_many_parts(lib, workspace, dim, dtype):
    run(lib, workspace, 1, 4, dim, 64, [20011], trees((12, "wide")), dtype, 64, False, seed=5)


def test_attend_tree_scales_and_equal_lengths(lib, workspace):
    run(lib, workspace, 2, 4, 128, 16, [40, 100], trees((6, "wide"), (6, "star")), BF16, 128, False, equal=True)
    run(lib, workspace, 1, 5, 64, 16, [40, 100], trees((30, "wide"), (18, "wide")), BF16, 64, False, ks=0.25, vs=3.7, scale=0.31)
    run(lib, workspace, 1, 3, 128, 16, [33], trees((20, "forest")), BF16, 0, False, scale=-0.05)


def test_attend_tree_peaked_and_flat_rows(lib, workspace):
    def edit(q):
        q[0] *= 40.0
        q[1] = 0.0
        q[2] *= 2.0 ** -60 if q.dtype != F16 else 2.0 ** -12
    for dtype in (F32, BF16):
        run(lib, workspace, 1, 4, 128, 16, [150], trees((24, "wide")), dtype, 0, False, edit=edit)


@pytest.mark.parametrize("grp,dtype", [(2, F32), (6, BF16)])
def test_attend_tree_nan_stays_with_the_rows_that_see_it(lib, workspace, grp, dtype):
    """A drafted token whose key or value reads as NaN: only its own subtree sees it."""
    for which in (0, 1):
        def poison(r, sk, sv):
            (sk, sv)[which][50 + 2, 0, 1] = 0x7F
        got, want = run(lib, workspace, 1, grp, 64, 16, [50], [[-1, 0, 0, 1, 2, 4, 0, 6]], dtype, 64, False, poison=poison)
        rows = want.isnan().flatten(1).any(1).tolist()
        assert rows == [False, False, True, False, True, True, False, False]


def test_attend_tree_chain_has_the_bits_of_kda_kv4_attend(lib, workspace):
    g = torch.Generator().manual_seed(2)
    ctx, lens = [200, 31, 64], [7, 1, 8]
    cache = ref.Cache([c + t for c, t in zip(ctx, lens)], 2, 128, 64, g)
    cos, sin = (x.cuda() for x in ref.tables(300, 128))
    for dtype in (BF16, F16):
        for window in (0, 40):
            q = torch.randn(sum(lens), 8, 128, generator=g).to(dtype).cuda()
            o, o2, st = torch.zeros_like(q), torch.zeros_like(q), i32([0])
            kw = dict(cu_seqlens=ragged(lens), max_t=8, cos=cos, sin=sin, window=window)
            common = (cache.pages.cuda(), cache.table.cuda(), i32(ctx), q)
            lib.kda_kv4_attend(*common, o, workspace, st, **kw)
            lib.kda_kv4_attend_tree(*common, tree_ref.masks(trees(*[(t, "chain") for t in lens])), o2, workspace, st, **kw)
            assert st.item() == 0
            # the same keys in the same order; only what a masked unit skips may differ
            assert (o.float() - o2.float()).abs().max() <= 2 * ref.half_step(dtype) * o.float().abs().max()


def test_attend_tree_bad_contexts_tables_and_pages(lib, workspace):
    heads, dim, page = 1, 64, 16
    pages = torch.full((4, heads, 1, 18 * dim), 0x11, dtype=torch.uint8, device="cuda")
    table = i32([[0, 1], [2, 3], [3, 1]])
    pars = trees((3, "star"), (3, "star"), (3, "star"))
    q = torch.randn(9, 2, dim, device="cuda")
    cos, sin = (t.cuda() for t in ref.tables(20, 32))

    def go(table, ctx, rot=True, cu=None):
        o, st = torch.full_like(q, 5.0), i32([0])
        lib.kda_kv4_attend_tree(pages, table, i32(ctx), q, tree_ref.masks(pars), o, workspace, st, cu_seqlens=None if cu is None else i32(cu),
                                max_t=3, cos=cos if rot else None, sin=sin if rot else None)
        torch.cuda.synchronize()
        assert not workspace[:2048].any()
        return st.item(), (o == 0).flatten(1).all(1).view(3, 3).all(1).tolist(), (o == 5).flatten(1).all(1).view(3, 3).all(1).tolist()

    assert go(table, [4, 4, 4])[0] == kda.KDA_OK
    assert go(table, [4, -1, 4])[:2] == (kda.KDA_ERR_ARG, [False, True, False])       # neither a context nor padding
    assert go(table, [4, -3, 4])[:2] == (kda.KDA_OK, [False, True, False])            # padding
    assert go(table, [4, 18, 4])[:2] == (kda.KDA_ERR_ARG, [False, True, False])       # past the rotation rows
    assert go(table, [4, 30, 4], rot=False)[:2] == (kda.KDA_ERR_ARG, [False, True, False])    # past the table
    bad = table.clone()
    bad[1, 0] = 4
    assert go(bad, [4, 4, 4])[:2] == (kda.KDA_ERR_SLOT_RANGE, [False, True, False])   # its only page: no key is seen
    st, zero, kept = go(table, [4, 4, 4], cu=[0, 3, 7, 9])                            # four tokens: that request is skipped
    assert st == kda.KDA_ERR_ARG
    # append: a context that is neither
    k, st, pg = torch.randn(9, heads, dim, device="cuda"), i32([0]), pages.clone()
    lib.kda_kv4_append_tree(pg, table, i32([4, -1, 4]), k, k, tree_ref.masks(pars), st, max_t=3, cos=cos, sin=sin)
    assert st.item() == kda.KDA_ERR_ARG and (pg != pages).flatten(1).any(1).tolist() == [True, False, False, True]


def test_attend_tree_padded_batch_leaves_the_rows_behind_it(lib, workspace):
    """Rows behind the last request's tokens stay as they are."""
    pages = torch.full((4, 1, 1, 18 * 64), 0x11, dtype=torch.uint8, device="cuda")
    q = torch.randn(9, 2, 64, device="cuda")
    o, st = torch.full_like(q, 5.0), i32([0])
    tree = torch.cat((tree_ref.masks(trees((3, "star"), (2, "star"))), torch.full((4,), -1, dtype=torch.int64, device="cuda")))
    lib.kda_kv4_attend_tree(pages, i32([[0], [1]]), i32([4, 4]), q, tree, o, workspace, st, cu_seqlens=i32([0, 3, 5]), max_t=3)
    assert st.item() == 0 and (o[5:] == 5).all() and not (o[:5] == 5).any()


def test_attend_tree_captured_beside_another_step(lib, workspace):
    """Two graphs on one workspace, replayed one after the other; then one on its own stream."""
    pars = trees((5, "wide"), (17, "wide"))
    g = torch.Generator().manual_seed(7)
    cache = ref.Cache([105, 317], 2, 128, 64, g)
    common = (cache.pages.cuda(), cache.table.cuda(), i32([100, 300]))
    tree, cu = tree_ref.masks(pars), ragged([5, 17])
    qs = [torch.randn(22, 8, 128, generator=g).to(BF16).cuda() for _ in range(2)]
    outs = [torch.zeros_like(qs[0]) for _ in range(4)]
    st = i32([0])
    for i in range(2):
        lib.kda_kv4_attend_tree(*common, qs[i], tree, outs[i], workspace, st, cu_seqlens=cu, max_t=17)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            lib.kda_kv4_attend_tree(*common, qs[i], tree, outs[2 + i], workspace, st, cu_seqlens=cu, max_t=17)
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert st.item() == 0 and torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])


# -- wide trees: the rows of a key/value head past 48 go to the tensor cores' other kernel --------------------------
WIDE = [("wide", 32, BF16, 128), ("wide", 32, F32, 128), ("forest", 24, F16, 64), ("chain", 24, BF16, 64), ("star", 40, F32, 64)]


@pytest.mark.parametrize("shape,grp,dtype,dim", WIDE)
@pytest.mark.parametrize("ctx", [0, 1, 63, 64, 65, 200])
def test_wide_tree_contexts_around_a_unit_of_keys(lib, workspace, shape, grp, dtype, dim, ctx):
    run(lib, workspace, 1, grp, dim, 16, [ctx], trees((3, shape)), dtype, dim, False, seed=ctx + grp)


@pytest.mark.parametrize("dtype,dim,inter", [(BF16, 128, True), (F32, 128, True), (F32, 128, False), (F16, 128, False), (BF16, 64, False), (F32, 64, True)])
def test_wide_tree_rows_around_a_tile(lib, workspace, dtype, dim, inter):
    """127, 128, 129 and 256 rows, and one head of many."""
    for t, grp in ((1, 127), (16, 8), (43, 3), (64, 4)):
        run(lib, workspace, 1, grp, dim, 32, [70], trees((t, "wide")), dtype, dim // 2, inter, seed=t)


@pytest.mark.parametrize("dtype,dim", [(BF16, 128), (F32, 128), (F16, 64), (BF16, 64)])
def test_wide_tree_rows_around_a_warp(lib, workspace, dtype, dim):
    """Tiles whose rows end within, at and behind a warp's 32: the other warps have none, and what rows that are not there
    hold is seen nowhere, also where a call before left NaN in every row."""
    def nan_rows(q):
        q[:] = float("nan")
    run(lib, workspace, 8, 128, dim, 16, [80], trees((1, "chain")), dtype, dim, False, seed=3, edit=nan_rows)
    run(lib, workspace, 2, 1, dim, 32, [70, 200, 5, 64, 0, 129, 33], trees((31, "wide"), (32, "chain"), (33, "wide"), (64, "forest"), (1, "chain"),
        (63, "star"), (2, "wide")), dtype, dim, False, seed=11)
    for grp in (65, 96, 97):
        run(lib, workspace, 1, grp, dim, 16, [190], trees((1, "chain")), dtype, dim, False, seed=grp)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_wide_trees_of_many_ragged_requests(lib, workspace, dtype):
    """40 requests and more, some empty, some padding: shares that begin and end anywhere in the list."""
    shapes = [(0 if r % 7 == 3 else 1 + (5 * r) % 9, ("wide", "chain", "star")[r % 3]) for r in range(43)]
    ctx = [-shapes[r][0] if r % 11 == 5 else (37 * r) % 150 for r in range(43)]
    run(lib, workspace, 1, 8, 64, 16, ctx, trees(*shapes), dtype, 64, False, seed=4)


def test_wide_tree_one_long_context_over_the_card(lib, workspace):
    run(lib, workspace, 1, 10, 128, 64, [20011], trees((7, "wide")), BF16, 128, False, seed=5)
    run(lib, workspace, 2, 26, 64, 64, [9000, 64], trees((2, "wide"), (5, "wide")), F32, 64, False, window=700, seed=6)


@pytest.mark.parametrize("dim,dtype", [(64, F32), (64, BF16), (128, BF16), (128, F16)])
def test_wide_tree_nan_stays_with_the_rows_that_see_it(lib, workspace, dim, dtype):
    """NaN in a drafted token's key or value, and in the value of a context token that a window hides from deep rows."""
    par = [-1, 0, 0, 1, 2, 4, 0, 6]
    for which in (0, 1):
        def poison(r, sk, sv):
            (sk, sv)[which][50 + 2, 0, 1] = 0x7F
        got, want = run(lib, workspace, 1, 16, dim, 16, [50], [par], dtype, 64, False, poison=poison)
        assert want.isnan().flatten(1).any(1).tolist() == [False, False, True, False, True, True, False, False]
    def early(r, sk, sv):
        sv[11, 0, dim // 16 - 1] = 0x7F
        sv[30, 0, 0] = 0x7F
    got, want = run(lib, workspace, 1, 16, dim, 16, [50], [par], dtype, 64, False, poison=early, window=40)
    assert want[:, :, dim - 1].isnan().all(1).tolist() == [True] + [False] * 7        # key 11 is in the root's window alone
    assert want[:, :, 0].isnan().all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_wide_tree_queries_far_from_one_and_not_finite(lib, workspace, dtype):
    def edit(q):
        q[0] *= 40.0
        q[1] = 0.0
        q[2] *= 2.0 ** -60
        q[3, 5, 7] = float("nan")
        q[4, 20, 0] = float("inf")
        q[5, 31, 9] = -float("inf")
    g = torch.Generator().manual_seed(3)
    cache = ref.Cache([157], 1, 128, 16, g)
    q = (torch.randn(7, 32, 128, generator=g) * 1.5).to(dtype)
    edit(q)
    o, st = torch.zeros(7, 32, 128, dtype=dtype, device="cuda"), i32([0])
    par = [ref_par for ref_par in trees((7, "wide"))]
    lib.kda_kv4_attend_tree(cache.pages.cuda(), cache.table.cuda(), i32([150]), q.cuda(), tree_ref.masks(par), o, workspace, st)
    bad = torch.zeros(7, 32, dtype=torch.bool)
    bad[3, 5] = bad[4, 20] = bad[5, 31] = True
    got = o.cpu().double()
    assert st.item() == 0 and torch.equal(got.isnan().all(-1), bad) and torch.equal(got.isnan().any(-1), bad)
    want, err, big, top = tree_ref.attend(cache, [150], par, torch.where(bad[..., None], torch.zeros_like(q), q), None, None, False)
    lim = ref.attend_tolerance(want, err, big, top, dtype, dtype != BF16)
    assert ((got - want).abs() <= lim)[~bad].all()


def test_wide_tree_bad_contexts_tables_and_pages(lib, workspace):
    dim = 64
    pages = torch.full((4, 1, 1, 18 * dim), 0x11, dtype=torch.uint8, device="cuda")
    table = i32([[0, 1], [2, 3], [3, 1]])
    pars = trees((3, "star"), (3, "star"), (3, "star"))
    q = torch.randn(9, 20, dim, device="cuda")
    cos, sin = (t.cuda() for t in ref.tables(20, 32))

    def go(table, ctx, rot=True, cu=None):
        o, st = torch.full_like(q, 5.0), i32([0])
        lib.kda_kv4_attend_tree(pages, table, i32(ctx), q, tree_ref.masks(pars), o, workspace, st, cu_seqlens=None if cu is None else i32(cu),
                                max_t=3, cos=cos if rot else None, sin=sin if rot else None)
        torch.cuda.synchronize()
        rows = lambda v: (o == v).flatten(1).all(1).view(3, 3).all(1).tolist()  # noqa: E731
        return st.item(), rows(0), rows(5)

    assert go(table, [4, 4, 4]) == (kda.KDA_OK, [False] * 3, [False] * 3)
    assert go(table, [4, -1, 4]) == (kda.KDA_ERR_ARG, [False, True, False], [False] * 3)
    assert go(table, [4, -3, 4]) == (kda.KDA_OK, [False, True, False], [False] * 3)
    assert go(table, [4, 18, 4]) == (kda.KDA_ERR_ARG, [False, True, False], [False] * 3)
    assert go(table, [4, 30, 4], rot=False) == (kda.KDA_ERR_ARG, [False, True, False], [False] * 3)
    assert go(table, [4, 2 ** 31 - 1, 4], rot=False) == (kda.KDA_ERR_ARG, [False, True, False], [False] * 3)
    for page in (4, -1, -2, 2 ** 31 - 1, -2 ** 31):
        bad = table.clone()
        bad[1, 0] = page
        assert go(bad, [4, 4, 4]) == (kda.KDA_ERR_SLOT_RANGE, [False, True, False], [False] * 3), page
    st, zero, kept = go(table, [4, 4, 4], cu=[0, 3, 7, 9])      # four tokens: that request is skipped
    assert st == kda.KDA_ERR_ARG and zero == [False] * 3
    # a page that is missing inside a context: its keys are not seen, the others are
    big = torch.randint(0, 256, (8, 1, 4, 18 * dim), generator=torch.Generator().manual_seed(1)).to(torch.uint8)
    big[..., 16 * dim:] = 0x30
    big = big.cuda()
    qs = torch.randn(3, 20, dim, device="cuda")
    outs = []
    for tab, ctx in ((i32([[0, 99, 2]]), 130), (i32([[0, 2]]), 66)):
        o, st = torch.zeros_like(qs), i32([0])
        lib.kda_kv4_attend_tree(big, tab, i32([ctx]), qs, tree_ref.masks(trees((3, "star"))), o, workspace, st)
        outs.append(o)
        assert st.item() == (kda.KDA_ERR_SLOT_RANGE if ctx == 130 else 0)
    assert (outs[0] - outs[1]).abs().max() <= 1e-5 * outs[1].abs().max()


@pytest.mark.parametrize("grp,dtype", [(4, BF16), (20, BF16), (20, F32)])
def test_attend_tree_reports_a_wait_that_runs_out(lib, workspace, grp, dtype):
    """Copies withheld by the test hook: the status, no fault, and the same workspace right again."""
    g = torch.Generator().manual_seed(2)
    cache = ref.Cache([203], 2, 64, 16, g)
    q, o = torch.randn(3, 2 * grp, 64, generator=g).to(dtype).cuda(), torch.full((3, 2 * grp, 64), 5.0, dtype=dtype, device="cuda")
    st, tree = i32([0]), tree_ref.masks(trees((3, "star")))
    common = (cache.pages.cuda(), cache.table.cuda(), i32([200]), q, tree, o, workspace, st)
    lib.kda_kv4_attend_tree(*common, flags=kda.KDA_LAUNCH_TEST_WITHHOLD_STATE)
    torch.cuda.synchronize()
    assert st.item() == kda.KDA_ERR_TIMEOUT and (o == 0).all()
    st.zero_()
    lib.kda_kv4_attend_tree(*common)
    want, err, big, top = tree_ref.attend(cache, [200], trees((3, "star")), q.cpu(), None, None, False)
    assert st.item() == 0
    assert ((o.cpu().double() - want).abs() <= ref.attend_tolerance(want, err, big, top, dtype, dtype != BF16)).all()
