"""The 4-bit paged cache at the ends of its ranges: kda_kv4_append and
kda_kv4_attend with counts, rows and pages where they can go wrong."""
import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

from test_gpu_kv4 import P, append_args, attend_args, cache_desc, run_attend

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
