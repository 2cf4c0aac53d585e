"""kda_step_tree and kda_conv_step_tree against fp64, with bounds derived in _tree_ref."""
import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

import _tree_ref as ref

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32


@pytest.fixture(scope="module")
def libs(built_libs):
    return {F32: kda.KdaLibrary(F32), F16: kda.KdaLibrary(F16)}


def ints(v, dtype=I32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def offsets(lens):
    cu = [0]
    for t in lens:
        cu.append(cu[-1] + t)
    return ints(cu)


# -- recurrence ------------------------------------------------------------------
class Step:
    """Inputs of one call: pars a parent list for each request."""

    def __init__(self, pars, hv, hqk, kd, vd, pool_dtype, dtype, learned=False, cols=None, seed=0, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.pars, self.lens = pars, [len(p) for p in pars]
        n, total = len(pars), sum(self.lens)
        self.max_t = max(self.lens)
        self.cols = self.max_t + 1 if cols is None else cols
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        slots = n * self.cols + spare
        self.pool = (0.5 * rand(slots, hv, kd, vd)).to(pool_dtype)
        self.table = torch.randperm(slots, generator=g)[: n * self.cols].to(I32).view(n, self.cols)
        self.accepted = torch.full((n,), self.cols, dtype=I32)
        self.q, self.k, self.v = rand(total, hqk, kd).to(dtype), rand(total, hqk, kd).to(dtype), rand(total, hv, vd).to(dtype)
        self.a, self.b = rand(total, hv, kd), rand(total, hv)
        self.a_log, self.dt_bias = (0.5 * rand(hv), 0.5 * rand(hv, kd)) if learned else (None, None)
        self.reset = None

    def run(self, lib, equal=False, stream=None, flags=0):
        c = lambda x: None if x is None else x.cuda()  # noqa: E731
        self.status = ints([0])
        pool = self.pool.cuda()
        o = torch.full(self.v.shape, 77.0, device="cuda")
        lib.kda_step_tree(pool, c(self.table), c(self.q), c(self.k), c(self.v), c(self.a), c(self.b), ref.masks(self.pars), o,
                          self.status, cu_seqlens=None if equal else offsets(self.lens), max_t=self.max_t, accepted=c(self.accepted),
                          reset=c(self.reset), a_log=c(self.a_log), dt_bias=c(self.dt_bias), stream=stream, flags=flags)
        torch.cuda.synchronize()
        return o.cpu(), pool.cpu()

    def check(self, o, pool, skip=()):
        """Every request's outputs and snapshots; what no request stores is untouched."""
        want = self.pool.clone()
        touched, at = set(), 0
        for r, t in enumerate(self.lens):
            sl = slice(at, at + t)
            at += t
            if t == 0:
                continue
            if r in skip:
                assert (o[sl] == 77.0).all()
                continue
            init = int(self.table[r, int(self.accepted[r]) - 1])
            if init < 0:
                assert (o[sl] == 0).all()
                continue
            S0 = self.pool[init].float()
            if self.reset is not None and self.reset[r]:
                S0 = torch.zeros_like(S0)
            oe, eo, S, es = ref.step(S0, self.pars[r], self.q[sl], self.k[sl], self.v[sl], self.a[sl], self.b[sl], self.a_log, self.dt_bias)
            assert ((o[sl].double() - oe).abs() <= eo + 1e-37).all(), r
            for j in range(t):
                s = int(self.table[r, j])
                if s < 0:
                    continue
                touched.add(s)
                lim = es[j] + (2.0 ** -11 * S[j].abs() + 2.0 ** -25 if pool.dtype == F16 else 0)
                assert ((pool[s].double() - S[j]).abs() <= lim * (1 + 2.0 ** -10)).all(), (r, j)
        rest = [s for s in range(pool.shape[0]) if s not in touched]
        assert torch.equal(pool[rest], want[rest])


@pytest.mark.parametrize("pool_dtype", [F32, F16])
@pytest.mark.parametrize("shapes,hv,hqk,kd,vd,dtype,learned", [
    ([(1, "chain")], 1, 1, 128, 128, BF16, False),
    ([(8, "wide")], 12, 12, 128, 128, BF16, False),
    ([(64, "wide")], 1, 1, 128, 128, BF16, False),
    ([(64, "chain")], 1, 1, 64, 48, F32, True),
    ([(17, "star"), (5, "forest"), (1, "chain"), (0, "chain"), (33, "wide")], 4, 2, 96, 80, F16, True),
    ([(9, "forest")] * 3, 3, 1, 16, 16, BF16, True),
    ([(7, "wide")] * 13, 6, 3, 112, 32, F32, False),
    ([(4, "wide")] * 40, 8, 8, 32, 128, F16, False),
    # enough column groups for one warp each, whole tiles and not
    ([(9, "wide")] * 8, 8, 4, 128, 128, BF16, False),
    ([(33, "forest")], 58, 58, 128, 128, F16, True),
    ([(13, "wide"), (64, "chain")], 50, 25, 64, 80, F32, False),
])
def test_step_tree_against_fp64(libs, pool_dtype, shapes, hv, hqk, kd, vd, dtype, learned):
    s = Step([ref.parents(t, k, i) for i, (t, k) in enumerate(shapes)], hv, hqk, kd, vd, pool_dtype, dtype, learned, seed=hv + kd)
    s.check(*s.run(libs[pool_dtype]))
    assert s.status.item() == 0


@pytest.mark.parametrize("pool_dtype", [F32, F16])
def test_step_tree_paths_do_not_depend_on_siblings(libs, pool_dtype):
    """Every root-to-leaf path gives the bits of the same tokens as a chain of their own."""
    lib = libs[pool_dtype]
    par = ref.parents(24, "wide", 5)
    s = Step([par], 4, 2, 128, 64, pool_dtype, BF16, True, seed=9)
    o, pool = s.run(lib)
    for path in ref.ancestors(par):
        c = Step([ref.parents(len(path), "chain")], 4, 2, 128, 64, pool_dtype, BF16, True)
        c.pool = s.pool[s.table[0, -1].item()].unsqueeze(0).repeat(len(path) + 2, 1, 1, 1)
        c.table = torch.arange(len(path) + 1, dtype=I32).view(1, -1)
        for name in ("q", "k", "v", "a", "b"):
            setattr(c, name, getattr(s, name)[path].contiguous())
        c.a_log, c.dt_bias = s.a_log, s.dt_bias
        oc, pc = c.run(lib)
        assert torch.equal(oc[-1], o[path[-1]])
        assert torch.equal(pc[len(path) - 1], pool[s.table[0, path[-1]].item()])


def test_step_tree_chain_is_close_to_kda_step(libs):
    """A chain: the same function as kda_step, two roundings apart; equal-length requests without offsets."""
    for pool_dtype, lim in ((F32, 1e-5), (F16, 2e-3)):
        s = Step([ref.parents(8, "chain")] * 3, 4, 4, 128, 128, pool_dtype, BF16, cols=9)
        o, pool = s.run(libs[pool_dtype], equal=True)
        s.check(o, pool)
        o2, p2, st = torch.zeros(24, 4, 128, device="cuda"), s.pool.cuda(), ints([0])
        libs[pool_dtype].kda_step(p2, s.table.cuda(), s.q.cuda(), s.k.cuda(), s.v.cuda(), s.a.cuda(), s.b.cuda(), o2, st, max_t=8,
                                  accepted=s.accepted.cuda())
        assert st.item() == 0
        assert (o2.cpu() - o).abs().max() <= 1e-5
        assert (p2.cpu().float() - pool.float()).abs().max() <= lim


def test_step_tree_resets_padding_and_columns_not_kept(libs):
    for pool_dtype in (F32, F16):
        s = Step([ref.parents(6, "wide", i) for i in range(5)], 2, 2, 64, 64, pool_dtype, BF16, seed=4)
        s.reset = torch.tensor([1, 0, 0, 1, 0], dtype=torch.uint8)
        s.table[1, -1] = -1                 # padding
        s.table[2, 3] = s.table[2, 0] = -5  # not kept
        s.check(*s.run(libs[pool_dtype]))
        assert s.status.item() == 0
        # the initial state's slot is a snapshot's too, as in a step that goes on from its own columns
        s.accepted = torch.tensor([1, s.cols, 2, 6, 3], dtype=I32)
        s.table[2, 1] = s.table[2, 6]
        s.check(*s.run(libs[pool_dtype]))
        assert s.status.item() == 0


def test_step_tree_bad_ids_and_offsets_are_reported_and_skipped(libs):
    lib = libs[F32]
    def fresh():
        return Step([ref.parents(3, "wide", i) for i in range(3)], 2, 1, 32, 32, F32, F32, seed=6)
    s = fresh()
    s.table[1, 2] = s.pool.shape[0]
    s.check(*s.run(lib), skip={1})
    assert s.status.item() == kda.KDA_ERR_SLOT_RANGE
    s = fresh()
    s.table[0, -1] = 1 << 30
    s.check(*s.run(lib), skip={0})
    assert s.status.item() == kda.KDA_ERR_SLOT_RANGE
    for bad in (0, 5, -3):
        s = fresh()
        s.accepted[2] = bad
        o, pool = s.run(lib)
        s.accepted[2] = 4
        s.check(o, pool, skip={2})
        assert s.status.item() == kda.KDA_ERR_ARG
    # offsets: decreasing, past total, more than max_t
    for cu in ([0, 3, 2, 9], [0, 3, 6, 10], [-1, 3, 6, 9], [0, 3, 7, 9]):
        s = fresh()
        o, st, pool = torch.full((9, 2, 32), 77.0, device="cuda"), ints([0]), s.pool.cuda()
        lib.kda_step_tree(pool, s.table.cuda(), s.q.cuda(), s.k.cuda(), s.v.cuda(), s.a.cuda(), s.b.cuda(), ref.masks(s.pars), o, st,
                          cu_seqlens=ints(cu), max_t=3, accepted=s.accepted.cuda())
        torch.cuda.synchronize()
        assert st.item() == kda.KDA_ERR_ARG


def test_step_tree_masks_with_other_bits(libs):
    """Bits above a token's own are ignored, its own counts as set."""
    s = Step([ref.parents(5, "wide", 2)], 2, 2, 32, 32, F32, F32, seed=8)
    o, pool = s.run(libs[F32])
    m = ref.masks(s.pars)
    for j in range(5):
        m[j] = (m[j] & ~(1 << j)) | -(1 << (j + 1))
    o2, p2, st = torch.zeros(5, 2, 32, device="cuda"), s.pool.cuda(), ints([0])
    libs[F32].kda_step_tree(p2, s.table.cuda(), s.q.cuda(), s.k.cuda(), s.v.cuda(), s.a.cuda(), s.b.cuda(), m, o2, st, accepted=s.accepted.cuda())
    assert st.item() == 0 and torch.equal(o2.cpu(), o) and torch.equal(p2.cpu(), pool)


# -- convolution -----------------------------------------------------------------
def run_conv(lib, pars, channels, width, dtype, silu=True, bias=True, length=None, seed=0, slots=None, accepted=None, reset=None,
             offset=0, equal=False):
    g = torch.Generator().manual_seed(seed)
    lens = [len(p) for p in pars]
    n, total = len(pars), sum(lens)
    length = width + 3 if length is None else length
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    window = rand(n + 2, length, channels).to(dtype)
    slots = torch.randperm(n + 2, generator=g)[:n].to(I32) if slots is None else torch.tensor(slots, dtype=I32)
    acc = torch.tensor([1 + r % (length - width + 2) for r in range(n)] if accepted is None else accepted, dtype=I32)
    x, w, b = rand(total, channels).to(dtype), rand(channels, width), rand(channels) if bias else None
    rst = None if reset is None else torch.tensor(reset, dtype=torch.uint8)
    # an offset moves x and y off a 16-byte boundary: the one-channel build
    hold = [torch.full((total * channels + offset,), 55.0, dtype=dtype, device="cuda") for _ in range(2)]
    xg, y = (h[offset:].view(total, channels) for h in hold)
    xg.copy_(x)
    wg, st = window.cuda(), ints([0])
    lib.kda_conv_step_tree(wg, slots.cuda(), xg, w.cuda(), ref.masks(pars), y, st, bias=None if b is None else b.cuda(),
                           cu_seqlens=None if equal else offsets(lens), max_t=max(lens), accepted=acc.cuda(),
                           reset=None if rst is None else rst.cuda(), silu=silu)
    torch.cuda.synchronize()
    assert torch.equal(wg.cpu(), window)
    got, at, bad = y.cpu().double(), 0, st.item()
    for r, (t, par) in enumerate(zip(lens, pars)):
        sl = slice(at, at + t)
        at += t
        if t == 0:
            continue
        slot, first = int(slots[r]), int(acc[r]) - 1
        if slot < 0:
            assert (got[sl] == 0).all()
        elif slot >= n + 2 or first < 0 or first + width - 1 > length:
            assert (got[sl] == 55).all() and bad
        else:
            hist = window[slot, first:first + width - 1]
            if reset is not None and reset[r]:
                hist = torch.zeros_like(hist)
            want, e = ref.conv(hist, par, x[sl], w, b, silu)
            lim = e + (0 if dtype == F32 else torch.finfo(dtype).eps / 2 * (want.abs() + e) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps)
            assert ((got[sl] - want).abs() <= lim).all(), r
    return bad


@pytest.mark.parametrize("shapes,channels,width,dtype,silu,bias,offset", [
    ([(8, "wide")], 4608, 4, BF16, True, True, 0),
    ([(64, "wide")] * 3, 512, 4, F16, True, False, 0),
    ([(1, "chain"), (0, "chain"), (13, "forest"), (64, "chain"), (21, "star")], 129, 3, F32, False, True, 0),
    ([(5, "wide"), (6, "forest")], 40, 8, BF16, True, True, 0),
    ([(5, "wide"), (6, "forest")], 44, 7, F32, True, True, 0),
    ([(9, "forest")], 64, 1, F16, True, True, 0),
    ([(9, "wide")] * 2, 64, 2, BF16, False, False, 1),
    ([(30, "forest")], 17, 6, F16, True, True, 3),
])
def test_conv_step_tree_against_fp64(libs, shapes, channels, width, dtype, silu, bias, offset):
    pars = [ref.parents(t, k, i) for i, (t, k) in enumerate(shapes)]
    assert run_conv(libs[F32], pars, channels, width, dtype, silu, bias, seed=channels, offset=offset) == 0


def test_conv_step_tree_padding_resets_and_refusals(libs):
    pars = [ref.parents(4, "wide", i) for i in range(4)]
    assert run_conv(libs[F32], pars, 64, 4, BF16, slots=[0, -1, 3, 2], reset=[1, 0, 0, 1], equal=True) == 0
    assert run_conv(libs[F32], pars, 64, 4, BF16, slots=[0, 6, 3, 2]) == kda.KDA_ERR_SLOT_RANGE
    for acc in ([1, 6, 1, 1], [0, 1, 1, 1], [1, 1, 1, -2 ** 31]):
        assert run_conv(libs[F32], pars, 64, 4, F32, accepted=acc, length=7) == kda.KDA_ERR_ARG
    st, y = ints([0]), torch.full((6, 64), 9.0, device="cuda")
    z = torch.zeros
    for cu in ([0, 4, 2], [0, 2, 7], [-1, 1, 2], [0, 5, 6]):
        st.zero_()
        libs[F32].kda_conv_step_tree(z(4, 3, 64, device="cuda"), ints([0, 1]), z(6, 64, device="cuda"), z(64, 4, device="cuda"),
                                     z(6, dtype=torch.int64, device="cuda"), y, st, cu_seqlens=ints(cu), max_t=4)
        assert st.item() == kda.KDA_ERR_ARG


@pytest.mark.parametrize("width,channels,dtype", [(4, 96, BF16), (3, 33, F16), (8, 64, F32)])
def test_conv_step_tree_chain_has_the_bits_of_kda_conv_step(libs, width, channels, dtype):
    g = torch.Generator().manual_seed(1)
    lens = [7, 1, 5]
    x = torch.randn(sum(lens), channels, generator=g).to(dtype).cuda()
    window = torch.randn(5, width + 7, channels, generator=g).to(dtype).cuda()
    w, b, slots, acc = torch.randn(channels, width, generator=g).cuda(), torch.randn(channels, generator=g).cuda(), ints([3, 0, 4]), ints([4, 9, 8])
    y, y2, st = torch.zeros_like(x), torch.zeros_like(x), ints([0])
    tree = ref.masks([ref.parents(t, "chain") for t in lens])
    # kda_conv_step also keeps old entries: its history ends where those L - T do, or behind
    libs[F32].kda_conv_step_tree(window, slots, x, w, tree, y, st, bias=b, cu_seqlens=offsets(lens), max_t=7, accepted=acc)
    libs[F32].kda_conv_step(window.clone(), slots, x, w, y2, st, bias=b, cu_seqlens=offsets(lens), max_t=7, accepted=acc)
    assert st.item() == 0 and torch.equal(y, y2)


def test_conv_step_tree_far_preactivations(libs):
    """SiLU from -200 to 200, infinities and NaN: the values of kda_conv_step."""
    x = torch.cat((torch.linspace(-200, 200, 4001), torch.tensor([-88.8, -87.4, 88.0, 1e-40, -1e-40, 0.0, float("inf"), float("-inf"), float("nan")])))
    x = x[: len(x) // 2 * 2].view(2, -1).repeat(2, 4)[:, :8016].contiguous().cuda()
    w, y, y2, st = torch.ones(x.shape[1], 1, device="cuda"), torch.zeros_like(x), torch.zeros_like(x), ints([0])
    window = torch.zeros(4, 1, x.shape[1], device="cuda")
    slots = ints([0, 1, 2, 3])
    libs[F32].kda_conv_step_tree(window, slots, x, w, torch.ones(4, dtype=torch.int64, device="cuda"), y, st)
    libs[F32].kda_conv_step(window, slots, x, w, y2, st)
    assert st.item() == 0 and torch.equal(y.view(torch.int32)[~y.isnan()], y2.view(torch.int32)[~y2.isnan()]) and torch.equal(y.isnan(), y2.isnan())
