"""The 4-bit paged cache: kda_kv4_append (bytes, bit for bit) and
kda_kv4_attend (against fp64, tolerance derived in _layer_ref)."""
import ctypes
import time

import pytest
import torch

import kda_linear_attention_gated_gb300 as kda
from kda_linear_attention_gated_gb300 import Kv4AppendArgs, Kv4AttendArgs, Kv4CacheDesc

import _layer_ref as ref
from _harness import lib_for

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
P = 0x7F0000100000


@pytest.fixture(scope="module")
def lib(built_libs):
    return kda.KdaLibrary(torch.float32)


# -- host checks (no GPU) -----------------------------------------------------
def cache_desc(**kw):
    d = dict(base=P, page_tokens=64, heads=2, dim=128, reserved=0, num_pages=8, page_stride=64 // 16 * 2 * 18 * 128, k_scale=1.0, v_scale=1.0)
    d.update(kw)
    return Kv4CacheDesc(*d.values())


def append_args(**kw):
    d = dict(n=3, total=3, max_t=1, dtype=kda.KDA_BF16, table_cols=4, rot_dim=128, interleaved=0, rope_rows=64, out_dtype=kda.KDA_BF16,
             reserved=0, k_stride=256, v_stride=256, cu_seqlens=None, page_table=P, ctx_len=P, k=P, v=P, cos=P, sin=P, k_out=None, v_out=None)
    d.update(kw)
    return Kv4AppendArgs(*d.values())


def attend_args(**kw):
    d = dict(n=3, total=3, max_t=1, dtype=kda.KDA_BF16, table_cols=4, rot_dim=128, interleaved=0, rope_rows=64, h_q=8, window=0, scale=0.0,
             reserved=0, q_stride=1024, cu_seqlens=None, page_table=P, ctx_len=P, q=P, cos=P, sin=P, o=P, workspace=P,
             workspace_bytes=kda.KDA_KV4_WORKSPACE_BYTES)
    d.update(kw)
    return Kv4AttendArgs(*d.values())


CACHE_BAD = [(dict(base=None), kda.KDA_ERR_NULL), (dict(base=P + 8), kda.KDA_ERR_ALIGN), (dict(page_tokens=24), kda.KDA_ERR_SHAPE),
             (dict(page_tokens=0), kda.KDA_ERR_SHAPE), (dict(heads=0), kda.KDA_ERR_SHAPE), (dict(dim=96), kda.KDA_ERR_SHAPE),
             (dict(num_pages=0), kda.KDA_ERR_SHAPE), (dict(page_stride=100), kda.KDA_ERR_SHAPE),
             (dict(page_stride=64 // 16 * 2 * 18 * 128 + 8), kda.KDA_ERR_ALIGN), (dict(k_scale=0.0), kda.KDA_ERR_ARG),
             (dict(v_scale=float("inf")), kda.KDA_ERR_ARG), (dict(v_scale=float("nan")), kda.KDA_ERR_ARG), (dict(reserved=1), kda.KDA_ERR_ARG)]
BOTH_BAD = [(dict(n=-1), kda.KDA_ERR_ARG), (dict(total=4), kda.KDA_ERR_SHAPE), (dict(dtype=9), kda.KDA_ERR_DTYPE_UNSUPPORTED),
            (dict(table_cols=0), kda.KDA_ERR_SHAPE), (dict(table_cols=1 << 26), kda.KDA_ERR_SHAPE), (dict(rot_dim=48), kda.KDA_ERR_SHAPE),
            (dict(rot_dim=160), kda.KDA_ERR_SHAPE), (dict(interleaved=2), kda.KDA_ERR_ARG), (dict(rope_rows=0), kda.KDA_ERR_SHAPE),
            (dict(page_table=None), kda.KDA_ERR_NULL), (dict(ctx_len=None), kda.KDA_ERR_NULL), (dict(cos=None), kda.KDA_ERR_NULL),
            (dict(ctx_len=P + 2), kda.KDA_ERR_ALIGN), (dict(reserved=1), kda.KDA_ERR_ARG)]


@pytest.mark.parametrize("which", ["append", "attend"])
def test_refusals_before_any_launch(lib, which):
    make, call = (append_args, lib.kda_kv4_append_raw) if which == "append" else (attend_args, lib.kda_kv4_attend_raw)
    for kw, code in CACHE_BAD:
        assert call(cache_desc(**kw), make(), P, None) == code, kw
    for kw, code in BOTH_BAD:
        assert call(cache_desc(), make(**kw), P, None) == code, kw
    assert call(cache_desc(), make(), None, None) == kda.KDA_ERR_NULL
    assert call(cache_desc(), make(), P, None, flags=kda.KDA_LAUNCH_PDL_EARLY_STATE) == kda.KDA_ERR_ARG
    own = [(dict(k_stride=255), kda.KDA_ERR_SHAPE), (dict(v_stride=260), kda.KDA_ERR_ALIGN), (dict(k=P + 8), kda.KDA_ERR_ALIGN),
           (dict(v=None), kda.KDA_ERR_NULL), (dict(k_out=P, out_dtype=5), kda.KDA_ERR_DTYPE_UNSUPPORTED), (dict(v_out=P + 4), kda.KDA_ERR_ALIGN)]
    if which == "attend":
        own = [(dict(h_q=3), kda.KDA_ERR_SHAPE), (dict(h_q=0), kda.KDA_ERR_SHAPE), (dict(total=51, max_t=17), kda.KDA_ERR_SHAPE),
               (dict(q_stride=1000), kda.KDA_ERR_SHAPE), (dict(window=-1), kda.KDA_ERR_ARG), (dict(scale=float("nan")), kda.KDA_ERR_ARG),
               (dict(workspace=None), kda.KDA_ERR_NULL), (dict(workspace_bytes=1 << 20), kda.KDA_ERR_SHAPE), (dict(o=P + 2), kda.KDA_ERR_ALIGN),
               (dict(q=None), kda.KDA_ERR_NULL)]
    for kw, code in own:
        assert call(cache_desc(), make(**kw), P, None) == code, kw
    hook = kda.KDA_OK if which == "attend" else kda.KDA_ERR_ARG       # the test hook is an option of the one that waits
    assert call(cache_desc(), make(n=0, total=0), P, None, flags=kda.KDA_LAUNCH_TEST_WITHHOLD_STATE) == hook
    # nothing to do: accepted without a launch
    assert call(cache_desc(), make(n=0, total=0), P, None) == kda.KDA_OK


def test_page_bytes(lib):
    assert lib.kda_kv4_page_bytes(128, 8, 128) == 128 * 8 * (2 * 64 + 2 * 8)
    for bad in ((8, 8, 128), (128, 0, 128), (128, 8, 32)):
        with pytest.raises(kda.KdaError) as e:
            lib.kda_kv4_page_bytes(*bad)
        assert e.value.code == kda.KDA_ERR_SHAPE
    out = ctypes.c_int64(0)
    assert lib.lib.kda_kv4_page_bytes(16, 1, 64, None) == kda.KDA_ERR_NULL
    assert lib.lib.kda_kv4_page_bytes(16, 1, 64, ctypes.byref(out)) == kda.KDA_OK and out.value == 18 * 64


def test_reference_encoder_takes_the_nearest_code():
    """The reference's own rounding against a search over all codes, ties at borders included."""
    x = torch.arange(-192, 193, dtype=F32).repeat(16, 1).T.reshape(-1)[:384 * 16].reshape(-1, 16) / 32
    x[:, 0] = 6.0      # scale 1 in every group
    c, s = ref.encode(x)
    got = ref.decode(c, s)
    signed = torch.cat((ref.E2M1, -ref.E2M1))
    best = (x.double().unsqueeze(-1) - signed).abs().amin(-1)
    assert torch.equal((x.double() - got).abs(), best)
    tie = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -2.5], dtype=F32)
    y = torch.zeros(1, 16)
    y[0, 0], y[0, 1:9] = 6.0, tie
    assert ref.decode(*ref.encode(y))[0, 1:9].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -2.0]


# -- append -------------------------------------------------------------------
def ragged(lens):
    cu = [0]
    for t in lens:
        cu.append(cu[-1] + t)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def append_reference(pages, table, page, ctx, lens, k, v, cos, sin, inter, ks=1.0, vs=1.0):
    """Bytes of the pages after the call, by the format's layout, and the stored values; token by token."""
    pages = pages.clone()
    kk, vv = k.float(), v.float()
    out = [torch.zeros(k.shape, dtype=torch.float64) for _ in range(2)]
    inv = [torch.tensor(1.0, dtype=F32) / torch.tensor(s, dtype=F32) for s in (ks, vs)]
    at = 0
    for r, t in enumerate(lens):
        for j in range(t):
            p = ctx[r] + j
            if p < 0:
                continue
            i = at + j
            x = kk[i:i + 1]
            if cos is not None:
                x = ref.rotate32(x, cos[p:p + 1], sin[p:p + 1], inter)
            ck, sk = ref.encode(x * inv[0])
            cv, sv = ref.encode(vv[i:i + 1] * inv[1])
            w = p % 16
            spread = lambda c: torch.cat((torch.zeros(w, *c.shape[1:], dtype=torch.uint8), c, torch.zeros(15 - w, *c.shape[1:], dtype=torch.uint8)))  # noqa: E731,B023
            ones = [torch.zeros_like(spread(c)) for c in (ck, sk, cv, sv)]
            ones[0][w], ones[1][w], ones[2][w], ones[3][w] = 0xF, 0xFF, 0xF, 0xFF
            mask = ref.pack(*ones)[:, 0]
            new = ref.pack(spread(ck), spread(sk), spread(cv), spread(sv))[:, 0]
            b = pages[table[r, p // page], :, p % page // 16]
            b[:] = (b & ~mask) | new
            out[0][i] = ref.decode(ck, sk)[0] * ks
            out[1][i] = ref.decode(cv, sv)[0] * vs
        at += t
    return pages, out


def run_append(lib, heads, dim, page, ctx, lens, dtype, rot, inter, seed=0, ks=1.0, vs=1.0, fused=False, x=None, out=True, equal=False, stream=None):
    g = torch.Generator().manual_seed(seed)
    total = sum(lens)
    ends = [max(0, c + t) for c, t in zip(ctx, lens)]
    cache = ref.Cache(ends, heads, dim, page, g)
    pages = cache.pages
    rows = max(1, max(ends))
    cos, sin = ref.tables(rows, rot) if rot else (None, None)
    if x is None:
        x = (torch.randn(total, 2 * heads + 3, dim, generator=g) * 3).to(dtype)
    if fused:   # slices of one projection's output: rows lie apart
        xg = x.cuda()
        k, v = xg[:, 1:1 + heads], xg[:, 1 + heads:1 + 2 * heads]
    else:
        k, v = x[:, 1:1 + heads].contiguous().cuda(), x[:, 1 + heads:1 + 2 * heads].contiguous().cuda()
    od = BF16 if dtype == F32 else dtype
    ko, vo = (torch.full((total, heads, dim), float("nan"), dtype=od, device="cuda") for _ in range(2)) if out else (None, None)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pg = pages.cuda()
    lib.kda_kv4_append(pg, cache.table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"), k, v, status,
                       cu_seqlens=None if equal else ragged(lens), max_t=max(lens),
                       cos=None if cos is None else cos.cuda(), sin=None if sin is None else sin.cuda(), interleaved=inter,
                       k_scale=ks, v_scale=vs, k_out=ko, v_out=vo, stream=stream)
    torch.cuda.synchronize()
    assert status.item() == 0
    want, vals = append_reference(pages, cache.table, page, ctx, lens, x[:, 1:1 + heads], x[:, 1 + heads:1 + 2 * heads], cos, sin, inter, ks, vs)
    assert torch.equal(pg.cpu(), want)
    if out:
        for got, w in ((ko, vals[0]), (vo, vals[1])):
            got = got.cpu().double()
            assert torch.equal(got.isnan(), w.isnan())
            fine = ~w.isnan()
            # code * scale has six significant bits: whole in 16-bit types; a global scale costs one fp32 and the output's rounding
            lim = 0.0 if ks == vs == 1.0 else 2.0 ** -24 + ref.half_step(od)
            assert ((got - w).abs()[fine] <= lim * (1 + 2.0 ** -20) * w.abs()[fine]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("heads,dim,page,ctx,lens,dtype,rot,inter", [
    (2, 128, 128, [0, 5, 127, 128, 300], [1, 1, 1, 1, 1], BF16, 128, False),
    (1, 64, 16, [0], [1], F32, 0, False),
    (3, 64, 48, [7, 0, -4, 30], [19, 33, 4, 1], F16, 32, True),
    (5, 128, 16, [15, -3], [18, 9], F32, 64, False),
    (8, 128, 64, [1000, 0], [9, 0], BF16, 128, True),
    (1, 128, 32, [3], [70], BF16, 96, False),
])
def test_append_is_bit_exact(lib, heads, dim, page, ctx, lens, dtype, rot, inter):
    run_append(lib, heads, dim, page, ctx, lens, dtype, rot, inter, seed=heads + dim)


@pytest.mark.gpu
def test_append_slices_scales_and_no_outputs(lib):
    run_append(lib, 4, 128, 64, [10, 40], [6, 6], BF16, 128, False, fused=True, equal=True)
    run_append(lib, 2, 64, 16, [10, 3], [6, 11], F16, 64, True, ks=0.37, vs=19.0)
    run_append(lib, 2, 128, 16, [0], [5], F32, 32, False, ks=64.0, out=False)


@pytest.mark.gpu
def test_append_zeros_borders_huge_and_not_finite(lib):
    """All-zero groups, values on borders between codes, subnormal scales, saturation, NaN and infinities."""
    x = torch.zeros(16, 5, 64)
    x[0] = 6.0
    x[0, :, 1:8] = torch.tensor([0.25, 0.75, -1.25, 1.75, 2.5, -3.5, 5.0])
    x[1], x[2], x[3] = 1e-3, -3e-5, 1e-7
    x[4], x[5] = 2688.0, 1e30
    x[5, :, 3:] = -4e4
    x[6, :, 5], x[7, :, 40], x[8, :, 63] = float("nan"), float("inf"), float("-inf")
    x[9] = -0.0
    x[10] = torch.arange(64) - 31.5
    x[11, :, ::16] = 0.013
    x[12] = 448 * 6 * 1.03
    x[13, :, 0] = 3.4e38
    run_append(lib, 1, 64, 16, [0], [16], F32, 0, False, x=x)
    run_append(lib, 1, 64, 16, [3], [16], F32, 64, False, x=torch.where(torch.isfinite(x), x, 0.0))


@pytest.mark.gpu
def test_append_bad_pages_and_positions_are_reported_and_skipped(lib):
    heads, dim, page = 1, 64, 16
    pages = torch.full((4, heads, 1, 18 * dim), 0x11, dtype=torch.uint8, device="cuda")
    x = torch.randn(3, heads, dim, device="cuda")
    good = torch.tensor([[0, 1], [2, 3], [3, 1]], dtype=torch.int32, device="cuda")
    cos, sin = (t.cuda() for t in ref.tables(20, 32))

    def go(table, ctx, rot=True):
        pg, st = pages.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        lib.kda_kv4_append(pg, table, torch.tensor(ctx, dtype=torch.int32, device="cuda"), x, x, st, cos=cos if rot else None, sin=sin if rot else None)
        torch.cuda.synchronize()
        changed = (pg != pages).flatten(1).any(1).tolist()
        return st.item(), changed

    assert go(good, [0, 0, 0]) == (kda.KDA_OK, [True, False, True, True])
    bad = good.clone()
    bad[1, 0] = 4
    assert go(bad, [0, 0, 0]) == (kda.KDA_ERR_SLOT_RANGE, [True, False, False, True])
    bad[1, 0] = -1
    assert go(bad, [0, 0, 0]) == (kda.KDA_ERR_SLOT_RANGE, [True, False, False, True])
    assert go(good, [0, 32, 0], rot=False) == (kda.KDA_ERR_ARG, [True, False, False, True])   # past the table
    assert go(good, [0, 20, 0]) == (kda.KDA_ERR_ARG, [True, False, False, True])              # past the rotation rows
    assert go(good, [0, 2 ** 31 - 1, 0]) == (kda.KDA_ERR_ARG, [True, False, False, True])
    assert go(good, [0, -2 ** 31, 0]) == (kda.KDA_OK, [True, False, False, True])             # padding


# -- attend -------------------------------------------------------------------
def run_attend(lib, heads, grp, dim, page, ctx, lens, dtype, rot, inter, window=0, seed=0, ks=1.0, vs=1.0, scale=None, fused=False, q_gain=1.5,
               ws=None, poison=None, edit=None, equal=False, flags=0):
    g = torch.Generator().manual_seed(seed)
    total, hq = sum(lens), heads * grp
    ends = [max(0, c + t) for c, t in zip(ctx, lens)]
    cache = ref.Cache(ends, heads, dim, page, g, poison=poison)
    cos, sin = ref.tables(max(1, max(ends)), rot) if rot else (None, None)
    x = (torch.randn(total, hq + 2, dim, generator=g) * q_gain).to(dtype)
    if edit is not None:
        edit(x)
    q = x[:, 1:1 + hq]
    qg = x.cuda()[:, 1:1 + hq] if fused else q.contiguous().cuda()
    o = torch.full((total, hq, dim), float("nan"), dtype=dtype, device="cuda")
    if ws is None:
        ws = torch.zeros(kda.KDA_KV4_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.kda_kv4_attend(cache.pages.cuda(), cache.table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"), qg, o, ws, status,
                       cu_seqlens=None if equal else ragged(lens), max_t=max(lens), cos=None if cos is None else cos.cuda(),
                       sin=None if sin is None else sin.cuda(), interleaved=inter, window=window, scale=scale, k_scale=ks, v_scale=vs, flags=flags)
    torch.cuda.synchronize()
    assert status.item() == 0
    assert not ws[:2048].any(), "the workspace's counters are not back at zero"
    want, err, big, top = ref.attend(cache, ctx, lens, q, cos, sin, inter, window, scale, ks, vs)
    split = dtype != BF16      # bf16 queries and probabilities are rounded to 11 bits, others keep remainders
    got = o.cpu().double()
    lim = ref.attend_tolerance(want, err, big, top, dtype, split)
    assert torch.equal(got.isnan(), want.isnan())
    bad = (got - want).abs() > lim
    assert not bad.any(), f"worst {((got - want).abs() / lim).nan_to_num(0).max():.3g} of the bound"
    return got, want


@pytest.mark.gpu
@pytest.mark.parametrize("heads,grp,dim,page,ctx,lens,dtype,rot,inter,window", [
    (1, 1, 128, 16, [0], [1], BF16, 0, False, 0),                          # a single key
    (2, 4, 128, 64, [15, 16, 300], [1, 1, 1], BF16, 128, False, 0),
    (2, 6, 64, 16, [37, 0, 130], [2, 1, 1], F16, 64, True, 0),
    (1, 8, 128, 128, [1000], [1], F32, 64, False, 0),
    (3, 5, 128, 48, [50, -2, 5, 9], [8, 2, 3, 0], BF16, 128, False, 0),    # ragged, a padding request, an empty one
    (1, 12, 64, 16, [-3, 70], [8, 8], BF16, 32, False, 0),                 # rows before position 0
    (2, 7, 64, 32, [200, 90], [16, 3], F32, 0, False, 0),
    (2, 2, 128, 16, [400, 33], [4, 4], F16, 128, False, 1),                # only itself
    (1, 16, 128, 64, [700, 20], [3, 3], BF16, 128, True, 100),
    (1, 33, 64, 16, [257], [2], BF16, 64, False, 37),
])
def test_attend_against_fp64(lib, heads, grp, dim, page, ctx, lens, dtype, rot, inter, window):
    run_attend(lib, heads, grp, dim, page, ctx, lens, dtype, rot, inter, window, seed=heads * grp + dim)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, F32)])
def test_attend_long_context_over_many_parts(lib, dim, dtype):
    """One request over the whole card: many parts to join."""
    run_attend(lib, 1, 4, dim, 64, [20011], [2], dtype, 64, False, seed=5)


@pytest.mark.gpu
def test_attend_slices_scales_and_equal_lengths(lib):
    run_attend(lib, 2, 4, 128, 16, [40, 100], [2, 2], BF16, 128, False, fused=True, equal=True)
    run_attend(lib, 1, 5, 64, 16, [40, 100], [3, 1], F32, 64, False, ks=0.25, vs=3.7, scale=0.31)
    run_attend(lib, 1, 3, 128, 16, [33], [1], F16, 0, False, scale=-0.05)


@pytest.mark.gpu
def test_attend_peaked_and_flat_rows(lib):
    """Scores of hundreds, all zero, and queries far from 1 (their fp16 scaling is a power of two a row)."""
    def edit(x):
        x[0] *= 40.0
        x[1] = 0.0
        x[2] *= 2.0 ** -60 if x.dtype != F16 else 2.0 ** -12
    run_attend(lib, 1, 4, 128, 16, [150], [4], F32, 0, False, edit=edit)
    run_attend(lib, 1, 4, 64, 16, [150], [4], BF16, 64, False, edit=edit)


@pytest.mark.gpu
@pytest.mark.parametrize("grp,dtype", [(2, F32), (6, BF16)])
def test_attend_nan_stays_with_the_rows_that_see_it(lib, grp, dtype):
    """A key or value group that reads as NaN: rows that do not see its token are untouched."""
    def key(r, sk, sv):
        sk[52, 0, 3] = 0x7F      # seen by the last two of four tokens
    got, want = run_attend(lib, 1, grp, 128, 16, [50], [4], dtype, 0, False, poison=key)
    assert want[:2].isfinite().all() and want[2:].isnan().all()

    def val(r, sk, sv):
        sv[52, 0, 3] = 0xFF
    got, want = run_attend(lib, 1, grp, 128, 16, [50], [4], dtype, 0, False, poison=val)
    assert want[:2].isfinite().all() and want[2:, :, 48:64].isnan().all() and want[2:, :, :48].isfinite().all()

    def early(r, sk, sv):
        sv[30, 0, 1], sk[31, 0, 0] = 0x7F, 0x7F
    got, want = run_attend(lib, 1, grp, 64, 16, [50], [4], dtype, 0, False, window=19, poison=early)   # tokens left of every window
    assert want.isfinite().all()
    got, want = run_attend(lib, 1, grp, 64, 16, [60], [4], dtype, 0, False, window=31, poison=early)   # in the first row's window only
    assert want[0].isnan().any() and want[2:].isfinite().all()


@pytest.mark.gpu
def test_attend_bad_pages_and_positions(lib):
    """A page outside the pool is not seen and reported; a request past its table gives zero rows; the others are right."""
    g = torch.Generator().manual_seed(3)
    cache = ref.Cache([64, 64, 64], 1, 64, 16, g)
    q = torch.randn(3, 2, 64, generator=g)
    ctx = [63, 63, 63]

    def go(table, ctx, **kw):
        o = torch.full(q.shape, float("nan"), device="cuda")
        ws = torch.zeros(kda.KDA_KV4_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        lib.kda_kv4_attend(cache.pages.cuda(), table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"), q.cuda(), o, ws, st, **kw)
        torch.cuda.synchronize()
        return o.cpu().double(), st.item()

    want, err, big, top = ref.attend(cache, ctx, [1, 1, 1], q, None, None, False)
    lim = ref.attend_tolerance(want, err, big, top, F32, True)
    bad = cache.table.clone()
    bad[1, 1] = cache.pages.shape[0]
    o, st = go(bad, ctx)
    assert st == kda.KDA_ERR_SLOT_RANGE
    keep = torch.cat((torch.arange(16), torch.arange(32, 64)))
    cache.k[1], cache.v[1] = cache.k[1][keep], cache.v[1][keep]
    w1 = ref.attend(cache, [63, 47, 63], [1, 1, 1], q, None, None, False)[0]
    assert ((o[[0, 2]] - want[[0, 2]]).abs() <= lim[[0, 2]]).all() and ((o[1] - w1[1]).abs() <= lim[1]).all()
    o, st = go(cache.table, [63, 64, 63])
    assert st == kda.KDA_ERR_ARG and (o[1] == 0).all() and ((o[[0, 2]] - want[[0, 2]]).abs() <= lim[[0, 2]]).all()
    cos, sin = (t.cuda() for t in ref.tables(64, 32))
    o, st = go(cache.table, [63, 63, 2 ** 31 - 1], cos=cos, sin=sin)
    assert st == kda.KDA_ERR_ARG and (o[2] == 0).all() and o[:2].isfinite().all()


@pytest.mark.gpu
def test_attend_is_deterministic_and_leaves_the_workspace_ready(lib):
    ws = torch.zeros(kda.KDA_KV4_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    kw = dict(heads=2, grp=4, dim=128, page=64, ctx=[4000, 10, 900], lens=[1, 1, 1], dtype=BF16, rot=128, inter=False, ws=ws)
    a, _ = run_attend(lib, **kw)
    b, _ = run_attend(lib, **kw)
    c, _ = run_attend(lib_for(torch.float16), **kw)
    assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.gpu
@pytest.mark.parametrize("ctx", [[63, 20], [5000, 20]])     # whole in their CTAs; in parts that meet in the workspace
def test_withheld_copies_time_out_and_leave_the_call_usable(lib, ctx):
    """Every wait for a block is bounded: with the copies withheld the call reports the timeout, and the next one is right."""
    ws = torch.zeros(kda.KDA_KV4_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    kw = dict(heads=1, grp=2, dim=128, page=16, ctx=ctx, lens=[1, 1], dtype=BF16, rot=0, inter=False, ws=ws)
    want, _ = run_attend(lib, **kw)
    g = torch.Generator().manual_seed(0)
    cache = ref.Cache([c + 1 for c in ctx], 1, 128, 16, g)
    q, st = torch.randn(2, 2, 128, dtype=BF16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full_like(q, float("nan"))
    t0 = time.monotonic()
    lib.kda_kv4_attend(cache.pages.cuda(), cache.table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"), q, o, ws, st,
                       flags=kda.KDA_LAUNCH_TEST_WITHHOLD_STATE)
    torch.cuda.synchronize()
    assert st.item() == kda.KDA_ERR_TIMEOUT and 0.9 <= time.monotonic() - t0 < 30
    assert not ws[:2048].any() and (o == 0).all()
    again, _ = run_attend(lib, **kw)
    assert torch.equal(want, again)


@pytest.mark.gpu
def test_offsets_past_31_bits(lib):
    """A pool of more than 2^32 bytes: pages at its far end are appended to and read."""
    heads, dim, page = 2, 128, 128
    num = (1 << 32) // lib.kda_kv4_page_bytes(page, heads, dim) + 40
    pages = torch.zeros(num, heads, page // 16, 18 * dim, dtype=torch.uint8, device="cuda")
    table = torch.tensor([[num - 1, num - 2]], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(1)
    k, v = torch.randn(140, heads, dim, generator=g), torch.randn(140, heads, dim, generator=g)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.kda_kv4_append(pages, table, torch.zeros(1, dtype=torch.int32, device="cuda"), k.cuda(), v.cuda(), st)
    q = torch.randn(1, heads, dim, generator=g)
    o, ws = torch.empty_like(q).cuda(), torch.zeros(kda.KDA_KV4_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    lib.kda_kv4_attend(pages, table, torch.tensor([139], dtype=torch.int32, device="cuda"), q.cuda(), o, ws, st)
    torch.cuda.synchronize()
    assert st.item() == 0 and not pages[:num - 2].any()
    cache = ref.Cache([0], heads, dim, page, g)
    cache.k, cache.v = [ref.decode(*ref.encode(k))], [ref.decode(*ref.encode(v))]
    want, err, big, top = ref.attend(cache, [139], [1], q, None, None, False)
    assert ((o.cpu().double() - want).abs() <= ref.attend_tolerance(want, err, big, top, F32, True)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("flags", [0, kda.KDA_LAUNCH_PDL])
def test_append_then_attend_in_a_graph_on_another_stream(lib, flags):
    """The two calls of a decode step, captured and replayed with growing contexts, against eager calls."""
    heads, grp, dim, page, n = 2, 4, 128, 16, 5
    g = torch.Generator().manual_seed(9)
    mk = lambda *s: torch.randn(*s, generator=g).to(BF16).cuda()  # noqa: E731
    table = torch.randperm(n * 8, generator=g).int().view(n, 8).cuda()
    cos, sin = (t.cuda() for t in ref.tables(128, dim))
    pages = [torch.zeros(n * 8, heads, 1, 18 * dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ws = [torch.zeros(kda.KDA_KV4_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda") for _ in range(2)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(n, dtype=torch.int32, device="cuda")
    k, v, q = mk(n, heads, dim), mk(n, heads, dim), mk(n, heads * grp, dim)
    o = [torch.empty_like(q) for _ in range(2)]

    def step(i, stream):
        lib.kda_kv4_append(pages[i], table, ctx, k, v, st, cos=cos, sin=sin, stream=stream, flags=flags)
        lib.kda_kv4_attend(pages[i], table, ctx, q, o[i], ws[i], st, cos=cos, sin=sin, stream=stream, flags=flags)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(1, side)          # warm: the module is loaded before the capture
    side.synchronize()
    pages[1].zero_()       # as pages[0]: contexts below start behind places that were never appended
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(1, side)
    start = torch.tensor([0, 15, 3, -1, 31], dtype=torch.int32, device="cuda")
    for i in range(40):
        ctx.copy_(start + i)
        for t in (k, v, q):
            t.copy_(mk(*t.shape))
        step(0, None)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o[0], o[1])
    assert torch.equal(pages[0], pages[1]) and st.item() == 0
