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


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [1, 2])
def test_gates_far_from_zero_in_fp32(lib, kind):
    """sigmoid and SiLU to the ends of fp32: e^x below -87 down to subnormal numbers and zero, one above.

    Bound: the fp32 work behind a gate's factor is 24 half steps (exponential, reciprocal, products), and a subnormal sigmoid is
    off by a last step, 2^-149, once for its exponential and once for the product; the gate and the row multiply that."""
    g = torch.tensor([0.0, -0.0, 1e-20, 20.0, 87.0, 200.0, 1e30, float("inf"), -20.0, -86.9, -87.1, -88.5, -95.0, -100.0, -103.5, -104.5, -150.0,
                      -1e4, -1e30, -3e38, float("-inf"), float("nan"), 5.0, -5.0])
    dim = g.numel()
    gate = g.view(1, 1, dim).repeat(2, 1, 1)
    o = torch.ones(2, 1, dim)
    o[1] = -3.0
    y = torch.empty(2, 1, dim, device="cuda")
    lib.kda_head_norm(o.cuda(), torch.ones(dim, device="cuda"), y, gate=gate.cuda(), activation=kind, eps=0.0)
    ro, x = torch.empty(2, dim, device="cuda"), torch.empty(2, dim, device="cuda")
    lib.kda_block_norm(torch.zeros(2, dim, device="cuda"), o[:, 0].cuda(), ro, w_post=torch.ones(dim, device="cuda"), gate=gate[:, 0].cuda(),
                       activation=kind, eps=0.0)
    want = ref.head_norm(o, torch.ones(dim), gate, kind, 0.0)
    lim = 25 * 2.0 ** -24 * want.abs() + 2.0 ** -148 * ((1 + gate.double().abs()) if kind == 2 else 1.0)
    for got in (y, ro.view(2, 1, dim)):
        got = got.cpu().double()
        assert torch.equal(got.isnan(), want.isnan())
        fine = want.isfinite()
        assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()])
        assert ((got - want).abs() <= lim)[fine].all(), ((got - want).abs() / lim).nan_to_num(0).view(2, -1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_sigmoid_of_every_16_bit_gate(lib, dtype):
    """The factor of a 16-bit gate, seen whole through an fp32 residual: within (1.25 |x| + 7) 2^-24 of the sigmoid where that is
    a normal fp32 number, nothing (less than 2^-125) below."""
    g = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(dtype)
    g = g[~g.isnan()].cuda()
    n = g.numel() // 8 * 8
    g = torch.cat((g[:n], g[-8:])).view(-1, 8)
    h, zero = torch.empty(g.shape, device="cuda"), torch.zeros(g.shape, device="cuda")
    lib.kda_block_norm(zero, torch.ones_like(g), h, gate=g, activation=1)
    x, h = g.cpu().double().flatten(), h.cpu().double().flatten()
    want = torch.sigmoid(x)
    normal = x >= -87.0
    assert ((h - want).abs() <= (1.25 * x.abs().clamp(max=90) + 7) * 2.0 ** -24 * want)[normal].all()
    assert (h[~normal].abs() <= 2.0 ** -125).all() and normal.sum() > 40000
