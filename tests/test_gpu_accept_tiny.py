"""kda_accept's test of a first draft, u q(x) < p(x), is exact also where the product is near or below fp32's smallest numbers."""
from fractions import Fraction

import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

import _tree_ref as ref

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32


@pytest.fixture(scope="module")
def lib(built_libs):
    return kda.KdaLibrary(F32)


def rows(exponent, dtype, seed, n=2000):
    """u, q and, for each, p on the product's fp32 place, a step below and a step above; whether u q < p, in exact arithmetic."""
    g = torch.Generator().manual_seed(seed)
    u = torch.rand(n, generator=g)
    q = ((1 + torch.rand(n, generator=g)).double() * 2.0 ** exponent).to(F32).to(dtype)
    exact = u.double() * q.double()             # 48 bits: exact in fp64
    near = exact.to(F32).to(dtype)
    step = lambda to: torch.nextafter(near, torch.tensor(to, dtype=dtype))  # noqa: E731
    p = torch.stack((near, step(0.0), step(1.0)))
    return u.repeat(3), q.repeat(3), p.flatten(), (exact.repeat(3) < p.flatten().double())


@pytest.mark.parametrize("exponent,dtype", [(-1, F32), (-60, F32), (-99, F32), (-105, F32), (-124, F32), (-130, F32), (-140, F32), (-149, F32),
                                            (-104, BF16), (-128, BF16), (-10, F16), (-20, F16)])
def test_first_drafts_next_to_their_border(lib, exponent, dtype):
    u, q, p, want = rows(exponent, dtype, 7 - exponent)
    n, vocab = len(u), 5
    for i in torch.randint(0, n, (20,), generator=torch.Generator().manual_seed(1)).tolist():      # the fp64 products are the rational ones
        assert want[i].item() == (Fraction(u[i].item()) * Fraction(q[i].item()) < Fraction(p[i].item()))
    P, Q = torch.zeros(2 * n, vocab, dtype=dtype), torch.zeros(2 * n, vocab, dtype=dtype)
    P[0::2, 3], Q[0::2, 3] = p, q
    P[:, 0] = 0.5
    pars = [[-1, 0]] * n
    tokens = torch.tensor([0, 3] * n, dtype=I32)
    us = torch.zeros(2 * n)
    us[1::2] = u
    out = [torch.full(s, 99, dtype=I32, device="cuda") for s in ((n,), (n,), (n, 2), (n,))]
    st = torch.zeros(1, dtype=I32, device="cuda")
    lib.kda_accept(P.cuda(), tokens.cuda(), us.cuda(), torch.full((n,), 0.5, device="cuda"), *out, st, q=Q.cuda(), tree=ref.masks(pars))
    assert st.item() == 0
    assert torch.equal(out[0].cpu(), 1 + want.int())
