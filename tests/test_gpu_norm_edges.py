"""kda_head_norm and kda_block_norm at the ends of their ranges."""
import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

import _layer_ref as ref

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def lib(built_libs):
    return kda.KdaLibrary(torch.float32)


@pytest.mark.gpu
def test_block_norm_of_the_most_rows_there_can_be(lib):
    """2^31 - 1 rows: the row after a CTA's last one is past 2^31, where a signed count would turn negative."""
    total = 2 ** 31 - 1
    r = torch.empty(total, 1, dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    r[:] = torch.randn(1 << 20, generator=g, device="cuda").to(BF16).repeat(1 << 11)[:total, None]
    x = torch.full_like(r, float("nan"))
    lib.kda_block_norm(r, None, None, w_pre=torch.full((1,), 0.75, device="cuda"), x=x, eps=0.5)
    for a in range(0, total, 1 << 27):
        want = r[a:a + (1 << 27)].double()
        want = 0.75 * want / torch.sqrt(want * want + 0.5)
        # one rounding to bf16 behind fp32 work of a few half steps
        bad = (x[a:a + (1 << 27)].double() - want).abs() > (ref.half_step(BF16) + 2.0 ** -19) * want.abs()
        assert not bad.any()
