"""The 4-bit paged cache at the ends of its ranges: kda_kv4_append and
kda_kv4_attend with counts, rows and pages where they can go wrong."""
import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

from test_gpu_kv4 import P, append_args, attend_args, cache_desc

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
