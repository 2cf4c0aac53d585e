"""The operators together: the example's hybrid stack, step by step against the
same model in fp64 (the recurrence's and the norms' formulas, attention over the
values that 4-bit blocks hold), and its captured step against the eager one."""
import os
import sys

import pytest
import torch

import _layer_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

SMALL = dict(n=3, layers=3, hidden=256, hv=2, dim=128, h_q=4, h_kv=2, page=16, max_len=64)


class Plain:
    """The stack in fp64 on the CPU, weights and bf16 activations at the same places as the library's inputs."""

    def __init__(self, stack):
        self.s = stack
        self.c = lambda t: t.detach().cpu().double()
        self.state = [torch.zeros(stack.n, stack.hv, stack.dim, stack.dim, dtype=torch.float64) for _ in stack.layers]
        self.keys = [[] for _ in stack.layers]
        self.t = 0

    def step(self, x):
        s, c = self.s, self.c
        n, d = s.n, s.dim
        bf = lambda t: t.to(torch.bfloat16).double()  # noqa: E731
        res = bf(x)
        h = bf(ref.rms(res, 1e-6) * c(s.first))
        for i, w in enumerate(s.layers):
            p = bf(h @ c(w["in"]).T)
            if w["attention"]:
                p = p.view(n, -1, d)
                cos, sin = c(s.cos)[self.t:self.t + 1], c(s.sin)[self.t:self.t + 1]
                q = ref.rotate32(p[:, :s.h_q], cos.expand(n, -1), sin.expand(n, -1), False)
                k = ref.rotate32(p[:, s.h_q:s.h_q + s.h_kv], cos.expand(n, -1), sin.expand(n, -1), False)
                hold = lambda v: ref.decode(*ref.encode(v.float()))  # noqa: E731
                self.keys[i].append((hold(k), hold(p[:, s.h_q + s.h_kv:])))
                K, V = (torch.stack([a[j] for a in self.keys[i]], 2).repeat_interleave(s.h_q // s.h_kv, 1) for j in (0, 1))
                o = torch.softmax((K @ q.unsqueeze(-1)).squeeze(-1) * d ** -0.5, -1).unsqueeze(-2) @ V
                o = bf(o.squeeze(-2))
            else:
                p = p.view(n, 4, s.hv, d)
                unit = lambda v: v / torch.sqrt((v * v).sum(-1, keepdim=True) + 1e-6)  # noqa: E731
                q, k, v = unit(p[:, 0]), unit(p[:, 1]), p[:, 2]
                a = bf(h @ c(w["decay"]).T).view(n, s.hv, d)
                b = torch.sigmoid(bf(h @ c(w["beta"]).T)).view(n, s.hv, 1, 1)
                S = self.state[i] * torch.sigmoid(-a).unsqueeze(-1)
                S = S + b * k.unsqueeze(-1) * (v - (S * k.unsqueeze(-1)).sum(-2)).unsqueeze(-2)
                self.state[i] = S
                o = (S * q.unsqueeze(-1)).sum(-2) * d ** -0.5
                o = bf(ref.rms(o, 1e-6) * c(w["norm"]) * torch.sigmoid(p[:, 3]))
            y = bf(o.reshape(n, -1) @ c(w["out"]).T)
            res, _, h = ref.block_norm(res, y, c(w["post"]), bf(h @ c(w["gate"]).T), 1, None, c(w["pre"]), 1.0, 0.5, 1e-6)
            h = bf(h)
        self.t += 1
        return h


@pytest.mark.gpu
@pytest.mark.usefixtures("built_libs")
def test_stack_follows_the_plain_model():
    """Both models round activations to bf16 at the same places, from values a few fp32 units apart: most roundings agree, some
    fall to the neighbour (2^-8 of the value at most, a small share), and a flipped 4-bit code moves one of many addends by a
    sixth.  Through three layers that stays below 2^-6 of the output's norm."""
    from hybrid_decode import HybridStack
    stack = HybridStack(**SMALL)
    plain = Plain(stack)
    g = torch.Generator().manual_seed(4)
    for _ in range(20):
        x = torch.randn(SMALL["n"], SMALL["hidden"], generator=g).to(torch.bfloat16)
        stack.x.copy_(x)
        got = stack.step().cpu().double()
        want = plain.step(x.double())
        assert torch.linalg.norm(got - want) <= 2.0 ** -6 * torch.linalg.norm(want)
    assert stack.status.item() == 0


@pytest.mark.gpu
@pytest.mark.usefixtures("built_libs")
def test_captured_step_is_the_eager_step():
    from hybrid_decode import HybridStack
    a, b = HybridStack(**SMALL), HybridStack(**SMALL)
    graph = b.capture()
    assert b.ctx.max().item() == 0
    g = torch.Generator().manual_seed(5)
    for _ in range(24):
        x = torch.randn(SMALL["n"], SMALL["hidden"], generator=g).to(torch.bfloat16)
        a.x.copy_(x)
        b.x.copy_(x)
        a.step()
        graph.replay()
        assert torch.equal(a.h, b.h)
    assert a.status.item() == 0 and b.status.item() == 0 and b.ctx.tolist() == [24] * SMALL["n"]
