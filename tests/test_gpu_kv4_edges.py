"""The 4-bit paged cache at the ends of its ranges: kda_kv4_append and
kda_kv4_attend with counts, rows and pages where they can go wrong."""
import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

import _layer_ref as ref
from test_gpu_kv4 import P, append_args, attend_args, cache_desc, ragged, run_attend

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
