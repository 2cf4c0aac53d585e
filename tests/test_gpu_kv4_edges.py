"""The 4-bit paged cache at the ends of its ranges: kda_kv4_append and
kda_kv4_attend with counts, rows and pages where they can go wrong."""
import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

import _layer_ref as ref
from test_gpu_kv4 import P, append_args, attend_args, cache_desc, ragged, run_append, run_attend

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def lib(built_libs):
    return kda.KdaLibrary(torch.float32)


# -- host checks (no GPU) -----------------------------------------------------
@pytest.mark.parametrize("which", ["append", "attend"])
def test_counts_next_to_31_bits_are_refused(lib, which):
    """Counts are rounded up in 32 bits on the device: those that would wrap are refused (no status word is given, so nothing
    could be launched either way)."""
    make, call = (append_args, lib.kda_kv4_append_raw) if which == "append" else (attend_args, lib.kda_kv4_attend_raw)
    for kw in (dict(n=2 ** 31 - 1), dict(total=2 ** 31 - 1), dict(n=2 ** 31 - 32), dict(total=2 ** 31 - 8)):
        assert call(cache_desc(), make(cu_seqlens=P, **kw), None, None) == kda.KDA_ERR_SHAPE, kw
    for kw in (dict(n=kda.KDA_KV4_MAX_COUNT), dict(total=kda.KDA_KV4_MAX_COUNT)):
        assert call(cache_desc(), make(cu_seqlens=P, **kw), None, None) == kda.KDA_ERR_NULL, kw


# -- attend -------------------------------------------------------------------
def many(n, seed):
    """Contexts and token counts of n requests: short ones, empty and padding ones, some rows before position 0, and a few long
    enough to be cut, at every place modulo 4 (a lane of the share search owns up to four of these requests)."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, 4, (n,), generator=g).tolist()
    ctx = torch.randint(0, 90, (n,), generator=g).tolist()
    for r in range(0, n, 7):
        ctx[r] = -lens[r]
    for r in range(3, n, 11):
        ctx[r], lens[r] = -1, 3
    for r in range(5, n, 9):
        ctx[r], lens[r] = 1500 + r, 2
    return ctx, lens


@pytest.mark.gpu
@pytest.mark.parametrize("n,heads,grp,dim,dtype,window", [
    (33, 4, 3, 128, BF16, 0), (64, 3, 2, 64, F16, 0), (64, 2, 8, 128, BF16, 41), (100, 4, 1, 64, F32, 0), (131, 2, 4, 128, BF16, 0), (97, 1, 5, 128, F32, 300),
])
def test_attend_of_more_requests_than_lanes(lib, n, heads, grp, dim, dtype, window):
    """Many parts a CTA, each with its own request, head and queries; shares that begin inside a lane's second or later request."""
    ctx, lens = many(n, seed=n + dim)
    run_attend(lib, heads, grp, dim, 32, ctx, lens, dtype, dim // 2, False, window, seed=n)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,grp,dim,lens,dtype", [(2, 4, 64, [8, 1, 3], BF16), (1, 3, 128, [2, 1, 1], F32), (3, 2, 64, [1, 1, 1], F16)])
def test_withheld_copies_of_every_build_time_out(lib, heads, grp, dim, lens, dtype):
    """Copies that never land, in parts that lie whole in a CTA and in ones that meet: zero rows, the timeout, a usable workspace."""
    ws = torch.zeros(kda.KDA_KV4_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    ctx = [3000, 40, 700]
    kw = dict(heads=heads, grp=grp, dim=dim, page=16, ctx=ctx, lens=lens, dtype=dtype, rot=0, inter=False, ws=ws)
    want, _ = run_attend(lib, **kw)
    cache = ref.Cache([c + t for c, t in zip(ctx, lens)], heads, dim, 16, torch.Generator().manual_seed(0))
    q = torch.randn(sum(lens), heads * grp, dim, device="cuda").to(dtype)
    o, st = torch.full_like(q, float("nan")), torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.kda_kv4_attend(cache.pages.cuda(), cache.table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"), q, o, ws, st,
                       cu_seqlens=ragged(lens), max_t=max(lens), flags=kda.KDA_LAUNCH_TEST_WITHHOLD_STATE)
    torch.cuda.synchronize()
    assert st.item() == kda.KDA_ERR_TIMEOUT and not ws[:2048].any() and (o == 0).all()
    again, _ = run_attend(lib, **kw)
    assert torch.equal(want, again)


@pytest.mark.gpu
def test_a_cache_with_dimensions_of_one_and_odd_strides(lib):
    """A dimension of size 1 says nothing about the layout, whatever its stride; real gaps between heads or blocks are refused."""
    size, st = 18 * 64, torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx, table = torch.full((1,), 5, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda")

    def append(pages, heads):
        x = torch.randn(1, heads, 64, generator=torch.Generator().manual_seed(2)).cuda()
        lib.kda_kv4_append(pages, table, ctx, x, x, st)
        torch.cuda.synchronize()
        return pages

    for num, heads, blocks in ((3, 1, 4), (3, 4, 1), (3, 1, 1), (1, 2, 2), (1, 1, 1)):
        want = append(torch.zeros(num, heads, blocks, size, dtype=torch.uint8, device="cuda"), heads)
        assert want.any()
        for odd in (7, size + 16):
            strides = list(want.stride())
            for d, n in enumerate(want.shape):
                if n == 1:
                    strides[d] = odd
            assert torch.equal(append(torch.zeros_like(want).as_strided(want.shape, strides), heads), want)
    # pages apart from each other are fine, as before
    wide = torch.zeros(3, 2 * 4 * size, dtype=torch.uint8, device="cuda")
    append(wide[:, :4 * size].view(3, 1, 4, size), 1)
    assert wide[0, :size].any() and not wide[:, size:].any() and not wide[1:].any()
    for bad in (torch.zeros(3, 2, 4, size, dtype=torch.uint8, device="cuda").transpose(1, 2), wide.view(3, 2, 4, size)[:, :, :2],
                torch.zeros(3, 2, 4, 2 * size, dtype=torch.uint8, device="cuda")[..., ::2]):
        with pytest.raises(ValueError):
            append(bad, bad.shape[1])
    assert st.item() == 0


def pages_of(k, v, page):
    """Pages [n, heads, page / 16, 18 dim] that hold fp32 k, v [tokens, heads, dim] from position 0 on, and the values they stand for."""
    t, heads, dim = k.shape
    pad = -t % page
    z = torch.zeros(pad, heads, dim)
    (ck, sk), (cv, sv) = ref.encode(torch.cat((k, z))), ref.encode(torch.cat((v, z)))
    blocks = ref.pack(ck, sk, cv, sv)
    pages = blocks.view(heads, -1, page // 16, 18 * dim).transpose(0, 1).contiguous()
    return pages, ref.decode(ck, sk)[:t], ref.decode(cv, sv)[:t]


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [19, 24, 26])
@pytest.mark.parametrize("dim,grp,dtype", [(128, 2, F32), (64, 2, F16), (64, 2, F32), (128, 2, BF16), (64, 12, BF16)])
def test_attend_behind_a_few_dominant_keys(lib, dim, grp, dtype, bits):
    """Sinks: keys that outweigh each of the others by about 2^bits, with values of zero in most channels, so that what the many
    others add stands alone.  Enough requests (on the same pages) that a warp works on thousands of keys behind a sink.

    Bound.  A probability is rounded to 2^-12 of it (with remainders 2^-22), or, where it is small, by an absolute 2^-35 (half of
    fp16's smallest step, 2^-25, with the maximum held at 2^10 or more).  Its exponent carries the score's errors.  The sums of a
    warp run over at most N / 16 mma (twice with remainders) of 17 addends, each off by 2^-24 of the sum of magnitudes; the sum of
    probabilities over N.  Then the output's rounding."""
    n, N, page, split = 400, 16384, 64, dtype != BF16
    g = torch.Generator().manual_seed(bits)
    k, v = torch.randn(N, 1, dim, generator=g), 1 + 0.3 * torch.randn(N, 1, dim, generator=g)
    k[:, 0, 0] = torch.tensor([-0.5, 0.0, 0.5])[torch.randint(0, 3, (N,), generator=g)]
    k[:, 0, 1] = 6.0                  # the group's scale is 1: channel 0 holds its values as they are
    sinks = torch.arange(8) * 32      # one in the first unit of each warp
    k[sinks, 0, 0] = 6.0
    v[sinks, 0, 16:] = 0.0
    pages, kv, vv = pages_of(k, v, page)
    q = torch.zeros(n, grp, dim)
    q[:, :, 0] = torch.tensor([1.0, 0.5, 0.75, 0.25]).repeat(3)[:grp]
    q = q.to(dtype)
    scale = bits * 0.6931471805599453 / 6
    o, st = torch.full((n, grp, dim), float("nan"), dtype=dtype, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(kda.KDA_KV4_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    lib.kda_kv4_attend(pages.cuda(), torch.arange(N // page, dtype=torch.int32, device="cuda").repeat(n, 1),
                       torch.full((n,), N - 1, dtype=torch.int32, device="cuda"), q.cuda(), o, ws, st, scale=scale)
    torch.cuda.synchronize()
    assert st.item() == 0
    s = torch.tensor(scale, dtype=F32).double() * q[0].double() @ kv[:, 0].T
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p /= p.sum(-1, keepdim=True)
    want, mag = p @ vv[:, 0], p @ vv[:, 0].abs()
    score = 2 * s.abs().amax() * 20 * 2.0 ** -24
    sums = (N / 16 * (2 if split else 1) * 17 + N) * 2.0 ** -24
    rel = 2 * torch.expm1(score) + (2.0 ** -21 if split else 2.0 ** -11) + sums
    lim = ref.half_step(dtype) * want.abs() + mag * rel + N * 2.0 ** -35 * vv.abs().max() * p.amax(-1, keepdim=True)
    if dtype == F16:
        lim = lim + 2.0 ** -25        # the output's own smallest step
    bad = (o.cpu().double() - want).abs() > lim
    assert not bad.any(), f"worst {((o.cpu().double() - want).abs() / lim).max():.3g} of the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("grp,lens,dtype,window,page", [(2, [1, 1], BF16, 100, 16), (4, [4, 1], F32, 100, 16), (3, [8, 2], BF16, 33, 48), (1, [2, 2], F16, 1, 32)])
def test_attend_window_with_released_pages(lib, grp, lens, dtype, window, page):
    """Pages whose keys lie left of every window were released (no page there): not an error, and not read."""
    heads, dim, ctx = 2, 64, [700, 300]
    g = torch.Generator().manual_seed(window)
    cache = ref.Cache([c + t for c, t in zip(ctx, lens)], heads, dim, page, g)
    for r, c in enumerate(ctx):
        gone = (c - window + 1) // page       # pages that end at or before the first query's first key
        assert gone > 0
        cache.table[r, :gone] = torch.tensor([-1, 2 ** 31 - 1], dtype=torch.int32).repeat(gone)[:gone]
    q = torch.randn(sum(lens), heads * grp, dim, generator=g).to(dtype)
    o, st = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(kda.KDA_KV4_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    args = (cache.pages.cuda(), cache.table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"), q.cuda(), o, ws, st)
    lib.kda_kv4_attend(*args, cu_seqlens=ragged(lens), max_t=max(lens), window=window)
    torch.cuda.synchronize()
    assert st.item() == kda.KDA_OK
    want, err, big, top = ref.attend(cache, ctx, lens, q, None, None, False, window)
    assert ((o.cpu().double() - want).abs() <= ref.attend_tolerance(want, err, big, top, dtype, dtype != BF16)).all()
    # one page more is a page that the first query needs
    args[1][0, (ctx[0] - window + 1) // page] = -1
    lib.kda_kv4_attend(*args, cu_seqlens=ragged(lens), max_t=max(lens), window=window)
    torch.cuda.synchronize()
    assert st.item() == kda.KDA_ERR_SLOT_RANGE


@pytest.mark.gpu
@pytest.mark.parametrize("dim,grp,dtype,rot", [(64, 2, F32, 0), (128, 2, BF16, 0), (64, 12, BF16, 0), (64, 2, F16, 32), (128, 2, F32, 128)])
def test_attend_queries_that_are_not_finite(lib, dim, grp, dtype, rot):
    """A query with an infinity (or of 1e37 and more) scores infinities or NaN with every key: its row is NaN by the softmax's
    definition, also where every score is minus infinity; other rows and requests stay right."""
    n, page = 6, 16
    for sign in (1.0, -1.0):
        k, v = sign * torch.ones(48, 1, dim), torch.randn(48, 1, dim, generator=torch.Generator().manual_seed(4))
        pages, kv, vv = pages_of(k, v, page)
        cos, sin = ref.tables(64, rot) if rot else (None, None)
        q = torch.randn(n, grp, dim, generator=torch.Generator().manual_seed(5))
        q[0, 0, 3], q[1, 1, dim - 1], q[2, 0, 5], q[3, 1, 0] = float("inf"), float("-inf"), float("nan"), float("-inf")
        if dtype != F16:
            q[4, 0, 1] = -2e38
        q = q.to(dtype)
        ctx = [0, 0, 40, 40, 9, 47]
        o, st = torch.zeros(n, grp, dim, dtype=dtype, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = torch.zeros(kda.KDA_KV4_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
        lib.kda_kv4_attend(pages.cuda(), torch.arange(3, dtype=torch.int32, device="cuda").repeat(n, 1), torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                           q.cuda(), o, ws, st, cos=None if cos is None else cos.cuda(), sin=None if sin is None else sin.cuda())
        torch.cuda.synchronize()
        assert st.item() == 0
        got = o.cpu().double()
        lost = ~(q.abs() < 1e37).all(-1)
        assert torch.equal(got.isnan(), lost.unsqueeze(-1).expand_as(got))
        cache = ref.Cache([0], 1, dim, page, torch.Generator())
        cache.k, cache.v = [kv] * n, [vv] * n
        want, err, big, top = ref.attend(cache, ctx, [1] * n, torch.where(lost.unsqueeze(-1), torch.zeros((), dtype=dtype), q), cos, sin, False)
        lim = ref.attend_tolerance(want, err, big, top, dtype, dtype != BF16)
        assert ((got - want).abs() <= lim)[~lost].all()


# -- append -------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("n,heads,dim,dtype,rot,inter,out", [(33, 2, 64, BF16, 64, False, True), (70, 3, 128, F16, 64, True, True), (131, 1, 64, F32, 0, False, False)])
def test_append_of_more_requests_than_lanes(lib, n, heads, dim, dtype, rot, inter, out):
    """The request of a token is found among more than 32, with empty and padding ones on both sides of every 32nd."""
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 4, (n,), generator=g).tolist()
    ctx = torch.randint(0, 50, (n,), generator=g).tolist()
    for r in (0, 30, 31, 32, 33, 62, 63, 64, 65, 95, 96, 127, 128):
        if r < n:
            lens[r] = 0
    for r in range(4, n, 13):
        lens[r], ctx[r] = 3, -3
    run_append(lib, heads, dim, 16, ctx, lens, dtype, rot, inter, seed=n, out=out)
    lens = [0] * 32 + [9] + [0] * (n - 33)     # every token behind the first 32 requests
    run_append(lib, heads, dim, 16, ctx, lens, dtype, rot, inter, seed=n, out=out)
