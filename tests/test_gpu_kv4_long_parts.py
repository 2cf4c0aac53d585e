"""Attention where one CTA works through a whole long context: as many requests as the card has places, all on the same pages.

The tensor cores round a sum towards zero at each addition.  A sum that n additions of like size make is off by half a step
(2^-24 of itself) of each at most, as it grows evenly; n is what one of the kernels adds up before it moves the sums on."""
import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

import _layer_ref as layer_ref
import _tree_ref as ref

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32
PAGE = 64


@pytest.fixture(scope="module")
def lib(built_libs):
    return kda.KdaLibrary(F32)


@pytest.fixture(scope="module")
def workspace():
    return torch.zeros(kda.KDA_KV4_TREE_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


_caches = {}


def cache(tokens, dim):
    """(pages, keys, values) of one request's tokens, one head; values of one sign, whose sums lose the same way throughout."""
    if (tokens, dim) not in _caches:
        g = torch.Generator().manual_seed(tokens + dim)
        full = -(-tokens // PAGE) * PAGE
        ck, sk = layer_ref.encode(torch.randn(full, 1, dim, generator=g))
        cv, sv = layer_ref.encode(torch.randn(full, 1, dim, generator=g).abs())
        pages = layer_ref.pack(ck, sk, cv, sv).view(1, -1, PAGE // 16, 18 * dim).transpose(0, 1).contiguous()
        _caches[tokens, dim] = pages, layer_ref.decode(ck, sk)[:tokens, 0], layer_ref.decode(cv, sv)[:tokens, 0]
    return _caches[tokens, dim]


def reference(ctx, k, v, q, dim):
    """As attend of _layer_ref, one head, all rows of a token at once."""
    t, grp, _ = q.shape
    o, err, big, top = torch.zeros(q.shape, dtype=torch.float64), *(torch.zeros(t, grp, dtype=torch.float64) for _ in range(3))
    for j in range(t):
        kk, vv, x = k[:ctx + j + 1], v[:ctx + j + 1], q[j].double()
        s = x @ kk.T * dim ** -0.5
        o[j] = torch.softmax(s, -1) @ vv
        err[j] = (x.abs() @ kk.abs().T * dim ** -0.5).amax(-1)
        big[j], top[j] = vv.abs().max(), s.abs().amax(-1)
    return o, err, big, top


def check(call, ctx, dim, dtype, t, grp, n, additions, gain=1.0):
    pages, k, v = cache(ctx + t, dim)
    g = torch.Generator().manual_seed(t * grp)
    q = (gain * torch.randn(t, grp, dim, generator=g)).to(dtype)
    table = torch.arange(pages.shape[0], dtype=I32).repeat(n, 1).cuda()
    qs = q.repeat(n, 1, 1).cuda()
    o, st = torch.full_like(qs, float("nan")), torch.zeros(1, dtype=I32, device="cuda")
    call(pages.cuda(), table, torch.full((n,), ctx, dtype=I32, device="cuda"), qs, o, st)
    assert st.item() == 0
    want, err, big, top = reference(ctx, k, v, q, dim)
    lim = layer_ref.attend_tolerance(want, err, big, top, dtype, dtype != BF16) + additions * 2.0 ** -24 * want.abs()
    got = o.cpu().double().view(n, t, grp, dim)
    assert ((got - want).abs() <= lim).all(), f"worst {((got - want).abs() / lim).max():.3g} of the bound"


@pytest.mark.parametrize("ctx,dim,dtype,t,grp", [
    (40000, 64, F32, 64, 2), (40000, 128, F32, 25, 2), (40000, 64, F16, 16, 4), (40000, 128, F16, 64, 2), (40000, 128, BF16, 64, 2),
    (131000, 64, F32, 64, 2), (131000, 128, F16, 64, 2), (131000, 64, BF16, 64, 1),
    # parts that end with, one unit ahead of and one behind a move of the sums (16 units of 64 keys)
    (1023, 64, F32, 64, 2), (1024, 64, F32, 64, 2), (1025, 64, F32, 64, 2), (2047, 128, F32, 64, 2), (2048, 128, F32, 64, 2), (2112, 128, F32, 64, 2),
    (4096, 64, F16, 64, 2), (4032, 64, F16, 64, 2), (16384, 128, BF16, 64, 2), (16320, 128, BF16, 64, 2),
])
def test_wide_trees(lib, workspace, ctx, dim, dtype, t, grp):
    additions = {F32: 16 * 8, F16: 64 * 8, BF16: 256 * 4}[dtype]
    n = 304
    tree = ref.masks([ref.parents(t, "chain")] * n)
    check(lambda pages, table, c, q, o, st: lib.kda_kv4_attend_tree(pages, table, c, q, tree, o, workspace, st, max_t=t), ctx, dim, dtype, t, grp, n,
          additions)
    assert not workspace[:2048].any()


@pytest.mark.parametrize("dim,dtype", [(64, F32), (128, F16), (128, BF16)])
def test_wide_trees_whose_maximum_keeps_rising(lib, workspace, dim, dtype):
    """Keys along the queries, longer and longer: sums that moved out meet later ones of other maxima."""
    ctx, t, grp, n = 9000, 16, 8, 304
    full = -(-(ctx + t) // PAGE) * PAGE
    g = torch.Generator().manual_seed(2)
    base = torch.randn(1, 1, dim, generator=g)
    gain = torch.linspace(0, 3, full).view(-1, 1, 1)
    ck, sk = layer_ref.encode(base * gain + 0.1 * torch.randn(full, 1, dim, generator=g))
    cv, sv = layer_ref.encode(torch.randn(full, 1, dim, generator=g))
    pages = layer_ref.pack(ck, sk, cv, sv).view(1, -1, PAGE // 16, 18 * dim).transpose(0, 1).contiguous()
    k, v = layer_ref.decode(ck, sk)[:ctx + t, 0], layer_ref.decode(cv, sv)[:ctx + t, 0]
    q = (torch.randn(t, grp, dim, generator=g) + base).to(dtype)
    want, err, big, top = reference(ctx, k, v, q, dim)
    qs = q.repeat(n, 1, 1).cuda()
    o, st = torch.full_like(qs, float("nan")), torch.zeros(1, dtype=I32, device="cuda")
    table = torch.arange(pages.shape[0], dtype=I32).repeat(n, 1).cuda()
    lib.kda_kv4_attend_tree(pages.cuda(), table, torch.full((n,), ctx, dtype=I32, device="cuda"), qs, ref.masks([ref.parents(t, "chain")] * n), o,
                            workspace, st, max_t=t)
    assert st.item() == 0
    lim = layer_ref.attend_tolerance(want, err, big, top, dtype, dtype != BF16) + 1024 * 2.0 ** -24 * big.unsqueeze(-1)
    got = o.cpu().double().view(n, t, grp, dim)
    assert ((got - want).abs() <= lim).all(), f"worst {((got - want).abs() / lim).max():.3g} of the bound"


# -- up to 48 query rows a head: kda_kv4_attend's kernel, for fp16 and fp32 queries 32 units of 32 keys a warp and sum --------
@pytest.mark.parametrize("ctx,dim,dtype,t,grp", [
    (131000, 64, F32, 1, 8), (131000, 128, F32, 2, 4), (131000, 128, F16, 1, 1), (40000, 64, F16, 2, 3), (131000, 128, BF16, 2, 4),
    # a warp's share at, one unit before and behind a move of the sums: eight warps (heads of 64) and six
    (8190, 64, F32, 1, 8), (8191, 64, F32, 1, 8), (8192, 64, F32, 1, 8), (8447, 64, F32, 1, 8), (16400, 64, F32, 1, 8),
    (6143, 128, F32, 1, 8), (6144, 128, F32, 1, 8), (6200, 128, F32, 1, 8), (6335, 128, F32, 1, 5), (12300, 128, F16, 1, 8),
])
@pytest.mark.parametrize("tree", [False, True])
def test_few_rows(lib, workspace, ctx, dim, dtype, t, grp, tree):
    n = 304
    masks = ref.masks([ref.parents(t, "chain")] * n)
    def call(pages, table, c, q, o, st):
        if tree:
            lib.kda_kv4_attend_tree(pages, table, c, q, masks, o, workspace, st, max_t=t)
        else:
            lib.kda_kv4_attend(pages, table, c, q, o, workspace, st, max_t=t)
    # bf16 queries: one sum a warp, at least six warps, 2 additions a unit
    additions = 32 * 4 if dtype != BF16 else 2 * ctx // 32 // 6
    check(call, ctx, dim, dtype, t, grp, n, additions)
    assert not workspace[:2048].any()


@pytest.mark.parametrize("gain", [2.0 ** -6, 0.0])
@pytest.mark.parametrize("dim,t,grp", [(64, 1, 8), (128, 2, 2)])
def test_few_rows_with_flat_scores(lib, workspace, dim, t, grp, gain):
    """Small queries: little but the sums' own errors is left of the bound."""
    call = lambda pages, table, c, q, o, st: lib.kda_kv4_attend(pages, table, c, q, o, workspace, st, max_t=t)  # noqa: E731
    check(call, 131000, dim, F32, t, grp, 304, 32 * 4, gain)


@pytest.mark.parametrize("dim,dtype", [(64, F32), (128, F16)])
def test_few_rows_whose_maximum_keeps_rising(lib, workspace, dim, dtype):
    ctx, t, grp, n = 30000, 2, 4, 304
    full = -(-(ctx + t) // PAGE) * PAGE
    g = torch.Generator().manual_seed(3)
    base = torch.randn(1, 1, dim, generator=g)
    gain = torch.linspace(0, 3, full).view(-1, 1, 1)
    ck, sk = layer_ref.encode(base * gain + 0.1 * torch.randn(full, 1, dim, generator=g))
    cv, sv = layer_ref.encode(torch.randn(full, 1, dim, generator=g))
    pages = layer_ref.pack(ck, sk, cv, sv).view(1, -1, PAGE // 16, 18 * dim).transpose(0, 1).contiguous()
    k, v = layer_ref.decode(ck, sk)[:ctx + t, 0], layer_ref.decode(cv, sv)[:ctx + t, 0]
    q = (torch.randn(t, grp, dim, generator=g) + base).to(dtype)
    want, err, big, top = reference(ctx, k, v, q, dim)
    o, st = torch.full((n * t, grp, dim), float("nan"), dtype=dtype, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
    table = torch.arange(pages.shape[0], dtype=I32).repeat(n, 1).cuda()
    lib.kda_kv4_attend(pages.cuda(), table, torch.full((n,), ctx, dtype=I32, device="cuda"), q.repeat(n, 1, 1).cuda(), o, workspace, st, max_t=t)
    assert st.item() == 0
    lim = layer_ref.attend_tolerance(want, err, big, top, dtype, True) + 128 * 2.0 ** -24 * big.unsqueeze(-1)
    got = o.cpu().double().view(n, t, grp, dim)
    assert ((got - want).abs() <= lim).all(), f"worst {((got - want).abs() / lim).max():.3g} of the bound"


def test_nan_and_windows_across_moves(lib, workspace):
    """A NaN value before the first move, seen by every row; and windows that begin behind it, which do not see it."""
    dim, ctx, n, grp = 64, 20000, 304, 4
    pages, k, v = (x.clone() for x in cache(ctx + 1, dim))
    byte = 17 * dim + (1 * 4 + 2) * 4        # the scale of token 4 of its block, channels 16 .. 31
    pages[0, 0, 0, byte] = 0x7F
    table = torch.arange(pages.shape[0], dtype=I32).repeat(n, 1).cuda()
    q = torch.randn(1, grp, dim, generator=torch.Generator().manual_seed(1))
    c = torch.full((n,), ctx, dtype=I32, device="cuda")
    tree = torch.ones(n, dtype=torch.int64, device="cuda")
    for rows in (grp, 16 * grp):
        qs = q.repeat(n, rows // grp, 1).cuda()
        for window in (0, 15000):
            o, st = torch.zeros_like(qs), torch.zeros(1, dtype=I32, device="cuda")
            lib.kda_kv4_attend_tree(pages.cuda(), table, c, qs, tree, o, workspace, st, window=window)
            assert st.item() == 0
            nan = o.isnan().cpu()
            assert nan[..., 16:32].all() == (window == 0) and not nan[..., :16].any() and not nan[..., 32:].any()
            if window:
                assert not nan.any()
