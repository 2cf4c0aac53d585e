"""The calls over trees with slots, pages and rows whose offsets pass 2^31 elements: the same values near and far are the same
results, bit for bit."""
import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

import _layer_ref as layer_ref
import _tree_ref as ref
from test_gpu_tree_step import Step

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32
FAR = (1 << 31) + 5


@pytest.fixture(scope="module")
def libs(built_libs):
    return {F32: kda.KdaLibrary(F32), F16: kda.KdaLibrary(F16)}


def ints(v, dtype=I32):
    return torch.tensor(v, dtype=dtype, device="cuda")


@pytest.mark.parametrize("hv", [1, 64])
def test_step_tree_slots(libs, hv):
    s = Step([ref.parents(9, "wide", i) for i in range(2)], hv, hv, 128, 128, F16, BF16, seed=5)
    o, pool = s.run(libs[F16])
    first = -(-FAR // (hv * 128 * 128))
    far = torch.empty(first + s.pool.shape[0], hv, 128, 128, dtype=F16, device="cuda")
    far[first:] = s.pool.cuda()
    far[:s.pool.shape[0]] = 7.0     # where offsets that wrap would go
    o2, st = torch.zeros_like(o, device="cuda"), ints([0])
    cu = ints([0, 9, 18])
    libs[F16].kda_step_tree(far, s.table.cuda() + first, s.q.cuda(), s.k.cuda(), s.v.cuda(), s.a.cuda(), s.b.cuda(), ref.masks(s.pars), o2, st,
                            cu_seqlens=cu, max_t=9, accepted=s.accepted.cuda())
    assert st.item() == 0 and torch.equal(o2.cpu(), o) and torch.equal(far[first:].cpu(), pool)
    assert (far[:s.pool.shape[0]] == 7).all()


def test_conv_step_tree_slots(libs):
    channels, g = 8192, torch.Generator().manual_seed(1)
    first = -(-FAR // (3 * channels))
    far = torch.zeros(first + 2, 3, channels, dtype=BF16, device="cuda")
    near = torch.randn(2, 3, channels, generator=g).to(BF16).cuda()
    far[first:] = near
    x, w = torch.randn(10, channels, generator=g).to(BF16).cuda(), torch.randn(channels, 4, generator=g).cuda()
    tree, out, st = ref.masks([ref.parents(5, "wide", i) for i in range(2)]), [], ints([0])
    for window, at in ((near, 0), (far, first)):
        y = torch.full_like(x, 9.0)
        libs[F32].kda_conv_step_tree(window, ints([at + 1, at]), x, w, tree, y, st, max_t=5)
        out.append(y)
    assert st.item() == 0 and torch.equal(*out)


@pytest.mark.parametrize("grp,dtype", [(2, F16), (16, BF16), (16, F32)])
def test_append_and_attend_tree_pages(libs, grp, dtype):
    lib, heads, dim, page, g = libs[F32], 8, 128, 64, torch.Generator().manual_seed(2)
    ctx = [150, 70]
    cache = layer_ref.Cache([c + 9 for c in ctx], heads, dim, page, g)
    size = heads * page // 16 * 18 * dim
    first = -(-FAR // size)
    far = torch.empty(first + cache.pages.shape[0], heads, page // 16, 18 * dim, dtype=torch.uint8, device="cuda")
    far[:8] = 0x7F                  # read back as NaN
    far[first:] = cache.pages.cuda()
    near = cache.pages.cuda()
    kv = torch.randn(2, 18, heads, dim, generator=g).to(dtype).cuda()
    q = torch.randn(18, heads * grp, dim, generator=g).to(dtype).cuda()
    tree, st, out = ref.masks([ref.parents(9, "wide", i) for i in range(2)]), ints([0]), []
    ws = torch.zeros(kda.KDA_KV4_TREE_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    for pages, at in ((near, 0), (far, first)):
        table = cache.table.cuda()
        table = torch.where(table >= 0, table + at, table)
        o = torch.zeros_like(q)
        lib.kda_kv4_append_tree(pages, table, ints(ctx), kv[0], kv[1], tree, st, max_t=9)
        lib.kda_kv4_attend_tree(pages, table, ints(ctx), q, tree, o, ws, st, max_t=9)
        out.append(o)
    assert st.item() == 0 and torch.equal(*out) and torch.equal(far[first:], near) and not out[0].isnan().any()
    assert (far[:8] == 0x7F).all()


@pytest.mark.parametrize("drawn", [True, False])
def test_accept_rows(libs, drawn):
    g = torch.Generator().manual_seed(3)
    total, vocab, stride = 18, 5003, 1 << 27
    pars = [ref.parents(9, "wide", i) for i in range(2)]
    rows = [torch.softmax(2 * torch.randn(total, vocab, generator=g), -1).to(BF16).cuda() for _ in range(2)]
    tokens, u, last = torch.randint(0, vocab, (total,), generator=g).to(I32).cuda(), torch.rand(total, generator=g).cuda(), torch.rand(2, generator=g).cuda()
    # likely drafts, so that the walks go down
    tokens[:] = (rows[0].float() / (rows[1].float() + 1e-3)).argmax(-1).to(I32)
    out = []
    hold = [torch.empty((total - 1) * stride + vocab, dtype=BF16, device="cuda") for _ in range(2)] if drawn else [torch.empty((total - 1) * stride + vocab, dtype=BF16, device="cuda")]
    for far in (False, True):
        p, q = rows if not far else [h.as_strided((total, vocab), (stride, 1)) for h in hold] + [None] * (2 - len(hold))
        if far:
            p.copy_(rows[0])
            if q is not None:
                q.copy_(rows[1])
        res = [torch.full(s, 99, dtype=I32, device="cuda") for s in ((2,), (2,), (2, 9), (2,))]
        st = ints([0])
        libs[F32].kda_accept(p, tokens, u, last, *res, st, q=q if drawn else None, tree=ref.masks(pars), max_t=9)
        assert st.item() == 0
        out.append(res)
    assert all(torch.equal(a, b) for a, b in zip(*out))
