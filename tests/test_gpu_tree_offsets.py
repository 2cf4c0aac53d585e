"""The calls over trees with token offsets that are not a batch's: what belongs to a refused request stays as it was (or gets
what a request without tokens gets), and the others are right."""
import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

import _layer_ref as layer_ref
import _tree_ref as ref
from test_gpu_kv4 import append_reference
from test_gpu_tree_step import Step

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32

# three requests of up to three tokens in nine rows: decreasing offsets, one past the end, a negative one, a request too long
OFFSETS = [([0, 3, 2, 9], {1, 2}), ([0, 3, 6, 10], {2}), ([-1, 3, 6, 9], {0}), ([0, 3, 7, 9], {1}), ([3, 2, 2, 5], {0}),
           ([0, 2 ** 31 - 1, -2 ** 31, 3], {0, 1, 2})]


@pytest.fixture(scope="module")
def libs(built_libs):
    return {F32: kda.KdaLibrary(F32), F16: kda.KdaLibrary(F16)}


@pytest.fixture(scope="module")
def workspace():
    return torch.zeros(kda.KDA_KV4_TREE_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


def ints(v, dtype=I32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def parents(masks, first, t):
    """Parents of a request's tokens, from the masks of its rows."""
    out = []
    for j in range(t):
        m = int(masks[first + j]) & ((1 << j) - 1)
        out.append(m.bit_length() - 1)
    return out


def valid(cu, bad, masks):
    """(request, first row, parents) of those that are taken."""
    return [(r, cu[r], parents(masks, cu[r], cu[r + 1] - cu[r])) for r in range(len(cu) - 1) if r not in bad]


MASKS = ref.masks([[-1, 0, 0], [-1, 0, 1], [-1, 0, 0]], device="cpu")


@pytest.mark.parametrize("cu,bad", OFFSETS)
@pytest.mark.parametrize("pool_dtype", [F32, F16])
@pytest.mark.parametrize("hv,kd,vd", [(2, 32, 48), (64, 128, 128)])
def test_step_tree(libs, pool_dtype, hv, kd, vd, cu, bad):
    s = Step([[-1, 0, 0]] * 3, hv, hv // 2, kd, vd, pool_dtype, BF16, seed=6)
    pool, o, st = s.pool.cuda(), torch.full(s.v.shape, 77.0, device="cuda"), ints([0])
    libs[pool_dtype].kda_step_tree(pool, s.table.cuda(), s.q.cuda(), s.k.cuda(), s.v.cuda(), s.a.cuda(), s.b.cuda(), MASKS.cuda(), o, st,
                                   cu_seqlens=ints(cu), max_t=3, accepted=s.accepted.cuda())
    assert st.item() == kda.KDA_ERR_ARG
    o, pool, want, rows = o.cpu(), pool.cpu(), s.pool.clone(), set()
    for r, at, par in valid(cu, bad, MASKS):
        sl = slice(at, at + len(par))
        rows |= set(range(at, at + len(par)))
        if not par:
            continue
        S0 = s.pool[s.table[r, int(s.accepted[r]) - 1].item()].float()
        oe, eo, S, es = ref.step(S0, par, s.q[sl], s.k[sl], s.v[sl], s.a[sl], s.b[sl])
        assert ((o[sl].double() - oe).abs() <= eo + 1e-37).all()
        for j in range(len(par)):
            slot = s.table[r, j].item()
            lim = es[j] + (2.0 ** -11 * S[j].abs() + 2.0 ** -25 if pool_dtype == F16 else 0)
            assert ((pool[slot].double() - S[j]).abs() <= lim * (1 + 2.0 ** -10)).all()
            want[slot] = pool[slot]
    assert torch.equal(pool, want)
    assert all((o[i] == 77).all() for i in range(9) if i not in rows)


@pytest.mark.parametrize("cu,bad", OFFSETS)
@pytest.mark.parametrize("dtype,channels", [(BF16, 64), (F32, 33)])
def test_conv_step_tree(libs, dtype, channels, cu, bad):
    g = torch.Generator().manual_seed(3)
    window = torch.randn(4, 3, channels, generator=g).to(dtype)
    x, w = torch.randn(9, channels, generator=g).to(dtype), torch.randn(channels, 4, generator=g)
    slots = [2, 0, 3]
    wg, y, st = window.cuda(), torch.full((9, channels), 55.0, dtype=dtype, device="cuda"), ints([0])
    libs[F32].kda_conv_step_tree(wg, ints(slots), x.cuda(), w.cuda(), MASKS.cuda(), y, st, cu_seqlens=ints(cu), max_t=3)
    assert st.item() == kda.KDA_ERR_ARG and torch.equal(wg.cpu(), window)
    y, rows = y.cpu(), set()
    for r, at, par in valid(cu, bad, MASKS):
        if not par:
            continue
        sl = slice(at, at + len(par))
        rows |= set(range(at, at + len(par)))
        want, e = ref.conv(window[slots[r]], par, x[sl], w, None, True)
        lim = e + (0 if dtype == F32 else torch.finfo(dtype).eps / 2 * (want.abs() + e) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps)
        assert ((y[sl].double() - want).abs() <= lim).all()
    assert all((y[i] == 55).all() for i in range(9) if i not in rows)


class Some:
    """Some requests of a cache."""

    def __init__(self, cache, which):
        self.heads, self.k, self.v = cache.heads, [cache.k[r] for r in which], [cache.v[r] for r in which]


@pytest.mark.parametrize("cu,bad", OFFSETS)
@pytest.mark.parametrize("grp,dim,dtype", [(2, 64, BF16), (20, 64, F32), (20, 128, BF16), (40, 128, F16)])
def test_attend_tree(libs, workspace, grp, dim, dtype, cu, bad):
    """On both sides of the wide trees' kernel."""
    g = torch.Generator().manual_seed(4)
    ctx, page = [40, 7, 100], 16
    cache = layer_ref.Cache([c + 3 for c in ctx], 2, dim, page, g)
    cos, sin = layer_ref.tables(110, dim)
    q = torch.randn(9, 2 * grp, dim, generator=g).to(dtype)
    o, st = torch.full(q.shape, 5.0, dtype=dtype, device="cuda"), ints([0])
    libs[F32].kda_kv4_attend_tree(cache.pages.cuda(), cache.table.cuda(), ints(ctx), q.cuda(), MASKS.cuda(), o, workspace, st, cu_seqlens=ints(cu),
                                  max_t=3, cos=cos.cuda(), sin=sin.cuda())
    assert st.item() == kda.KDA_ERR_ARG
    assert not workspace[:2048].any()
    ok = [v for v in valid(cu, bad, MASKS) if v[2]]
    rows = [i for _, at, par in ok for i in range(at, at + len(par))]
    o = o.cpu()
    assert all((o[i] == 5).all() for i in range(9) if i not in rows)
    if rows:
        want, err, big, top = ref.attend(Some(cache, [r for r, _, _ in ok]), [ctx[r] for r, _, _ in ok], [par for _, _, par in ok], q[rows], cos, sin, False)
        assert ((o[rows].double() - want).abs() <= layer_ref.attend_tolerance(want, err, big, top, dtype, dtype != BF16)).all()


@pytest.mark.parametrize("cu,bad", OFFSETS[:4])
def test_append_tree(libs, cu, bad):
    """(Offsets that leave rows to no request are kda_kv4_append's: those rows are refused one by one.)"""
    g = torch.Generator().manual_seed(5)
    ctx, page, heads, dim = [40, 7, 100], 16, 2, 64
    cache = layer_ref.Cache([c + 3 for c in ctx], heads, dim, page, g)
    cos, sin = layer_ref.tables(110, dim)
    x = torch.randn(2, 9, heads, dim, generator=g).to(BF16)
    pages, st = cache.pages.cuda(), ints([0])
    libs[F32].kda_kv4_append_tree(pages, cache.table.cuda(), ints(ctx), x[0].cuda(), x[1].cuda(), MASKS.cuda(), st, cu_seqlens=ints(cu), max_t=3,
                                  cos=cos.cuda(), sin=sin.cuda())
    assert st.item() == kda.KDA_ERR_ARG
    want = cache.pages
    for r, at, par in valid(cu, bad, MASKS):
        sl = slice(at, at + len(par))
        pos = [ctx[r] + len(p) - 1 for p in ref.ancestors(par)]
        k = layer_ref.rotate32(x[0, sl].float(), cos[pos], sin[pos], False)
        want, _ = append_reference(want, cache.table[r:r + 1], page, [ctx[r]], [len(par)], k, x[1, sl], None, None, False)
    assert torch.equal(pages.cpu(), want)


@pytest.mark.parametrize("cu,bad", OFFSETS)
@pytest.mark.parametrize("drawn", [True, False])
def test_accept(libs, drawn, cu, bad):
    g = torch.Generator().manual_seed(6)
    p = torch.softmax(2 * torch.randn(9, 61, generator=g), -1)
    q = torch.softmax(2 * torch.randn(9, 61, generator=g), -1) if drawn else None
    tokens, u, last = torch.randint(0, 61, (9,), generator=g).to(I32), torch.rand(9, generator=g), torch.rand(3, generator=g)
    out = [torch.full(s, 99, dtype=I32, device="cuda") for s in ((3,), (3,), (3, 3), (3,))]
    st = ints([0])
    libs[F32].kda_accept(p.cuda(), tokens.cuda(), u.cuda(), last.cuda(), *out, st, q=None if q is None else q.cuda(), tree=MASKS.cuda(),
                         cu_seqlens=ints(cu), max_t=3)
    assert st.item() == kda.KDA_ERR_ARG
    accepted, node, path, token = (t.tolist() for t in out)
    for r in bad:
        assert (accepted[r], node[r], token[r], path[r]) == (0, 0, -1, [-1] * 3)
    for r, at, par in valid(cu, bad, MASKS):
        if not par:
            assert (accepted[r], node[r], token[r], path[r]) == (0, 0, -1, [-1] * 3)
            continue
        sl = slice(at, at + len(par))
        want, nxt = ref.accept(p[sl], None if q is None else q[sl], tokens[sl], par, u[sl], last[r])
        assert path[r] == [at + i for i in want] + [-1] * (3 - len(want))
        assert (accepted[r], node[r], token[r]) == (len(want), want[-1] + 1, nxt)
