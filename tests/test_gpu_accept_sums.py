"""kda_accept next to its borders: draws and tests whose sides lie as near each other as the sums' bound allows.

The bound of a sum (and of a side of a test) over vocab entries, relative to the magnitudes added: (160 + vocab / 256)
2^-48, from u = 2^-24 and at most 5 u^2 a sum of two pairs of floats:
  a lane's chain      a step of up to four (16-bit types; two of fp32) weights without a renormalisation adds at most 32 (12) u^2
                      where the weights are pairs themselves: vocab / 16384 (8192) steps, so vocab / 512 u^2
  the cluster's sum   two chains, 5 + 6 levels of a tree: 60 u^2
  the draw            two levels of 5 and up to 8 parts, the difference, the product with u_last: 85 u^2; a thread's chain of
                      vocab / (16384 VE) vectors of VE weights, at most 96 (32) u^2 each, and its second look, a sum of two
                      pairs a weight, vocab / 16384 of them: vocab / 750 u^2
Cases keep a distance of twice that from their border, on both sides."""
from fractions import Fraction

import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32


@pytest.fixture(scope="module")
def lib(built_libs):
    return kda.KdaLibrary(F32)


def bound(vocab):
    return Fraction(160 + vocab // 256, 1 << 48)


def power(x):
    """The lowest power of two at or above x."""
    e = 0
    while Fraction(2) ** e >= x:
        e -= 1
    return 2.0 ** (e + 1)


def call(lib, p, q, tokens, u, u_last, tree):
    """One request's tokens a tree; (accepted, token)."""
    t = p.shape[0]
    c = lambda v, d: torch.tensor(v, dtype=d, device="cuda")  # noqa: E731
    out = [torch.full(s, 99, dtype=I32, device="cuda") for s in ((1,), (1,), (1, t), (1,))]
    st = c([0], I32)
    lib.kda_accept(p, c(tokens, I32), c(u, F32), c([u_last], F32), *out, st, q=q, tree=c(tree, torch.int64))
    torch.cuda.synchronize()
    assert st.item() == 0
    return out[0].item(), out[3].item()


def flat_tail(log_vocab):
    """A weight whose running sum behind 1 in plain fp32 loses nearly half a step with every second addition of a lane's
    2^(log_vocab - 12), always to the same side."""
    k = log_vocab - 13
    return ((1 << 23) + (1 << (k - 1)) - 1) * 2.0 ** -48


def halves(log_vocab, at, left):
    """A row whose two halves differ by `gap` alone: 1 and a flat tail, and the tail and 1 in 4096 pieces; the lower half is
    the heavier one if `left`.  (row, the border)"""
    h = (1 << (log_vocab - 1)) - 4096
    x = flat_tail(log_vocab)
    vocab = 2 * h + 4096 + 3
    whole = 2 * (1 + h * Fraction(x))
    gap = power(2 * 2 * bound(vocab) * whole)       # the border lies half of it away
    assert gap < x / 4
    row = torch.full((vocab,), x, device="cuda")
    row[0] = gap if left else 0.0
    row[1 + at] = 1.0
    border = 1 + h + 1
    row[border + h:border + h + 4096] = 2.0 ** -12
    row[vocab - 1] = 0.0 if left else gap
    return row, border


@pytest.mark.parametrize("left", [True, False])
@pytest.mark.parametrize("at", [0, 4321, -1, -77])
@pytest.mark.parametrize("log_vocab", [18, 20, 22, 24, 25])
@pytest.mark.parametrize("form", ["alone", "drawn", "given"])
def test_draws_next_to_a_border_of_many_weights(lib, form, log_vocab, at, left):
    """u_last is 1/2: the token on the heavier half's side of the border, however long the row."""
    row, border = halves(log_vocab, at if at >= 0 else (1 << (log_vocab - 1)) - 4096 + at, left)
    want = border - 1 if left else border
    if form == "alone":
        assert call(lib, row[None], None, [0], [0.0], 0.5, [1]) == (1, want)
        return
    # a draft of no weight is rejected first, and the sum is over what it leaves
    none = int(torch.nonzero(row == 0)[0])
    p, q = torch.stack((row, row)), None
    if form == "drawn":
        q = torch.zeros_like(p)
        q[:, none] = 1.0
    assert call(lib, p, q, [0, none], [0.0, 0.0], 0.5, [1, 3]) == (1, want)


@pytest.mark.parametrize("log_vocab", [25, 27])
def test_draws_from_equal_weights(lib, log_vocab):
    """Every sum of these weights has at most 46 bits, and so have u_last times their sum and its border: no rounding."""
    vocab = 1 << log_vocab
    row = torch.full((1, vocab), ((1 << (45 - log_vocab)) + 3) * 2.0 ** -45, device="cuda")
    for at in (0, 1, vocab // 3 & ~63, vocab // 2, vocab - 64):
        u = at / vocab
        assert torch.tensor(u, dtype=F32).item() == u
        assert call(lib, row, None, [0], [0.0], u, [1]) == (1, at)      # the sum has to pass u_last: on the border the next


@pytest.mark.parametrize("more", [True, False])
@pytest.mark.parametrize("log_vocab", [18, 20, 22, 24, 25])
def test_the_second_draft_next_to_its_border(lib, log_vocab, more):
    """u q(x) Z against W(x) for Z the sum of a long row's rest: 1/4 (S + a) against a, S within twice the bound of 3 a."""
    vocab = (1 << log_vocab) + 5
    x, n = flat_tail(log_vocab) / 4, 1 << log_vocab
    S = Fraction(1, 4) + (n - 1) * Fraction(x)
    a = Fraction(-(-S.numerator * (1 << 24) // (3 * S.denominator)), 1 << 24)
    gap = power(2 * bound(vocab) * 4 * a * 2)
    p = torch.full((3, vocab), x, device="cuda")
    p[:, 0] = 0.25
    # what is missing from 3 a (and the gap, to one side) in three weights, exactly
    left, parts = 3 * a + Fraction(gap) * (1 if more else -1) - S + 64 * Fraction(x), []
    p[:, 1:65] = 0.0        # of 64 weights of the tail, so that it is positive
    for _ in range(3):
        f = torch.tensor(float(left), dtype=F32)
        if Fraction(f.item()) > left:
            f = torch.nextafter(f, torch.tensor(0.0))
        parts.append(f.item())
        left -= Fraction(f.item())
    assert left == 0 and min(parts) >= 0
    p[:, n:n + 3] = torch.tensor(parts, device="cuda")
    x1, x2 = n + 3, n + 4
    q = torch.zeros_like(p)
    q[:, x1] = q[:, x2] = 0.5
    p[:, x1], p[:, x2] = 0.0, 0.5 + float(a)
    assert Fraction(p[0, x2].item()) == a + Fraction(1, 2)
    got, _ = call(lib, p, q, [0, x1, x2], [0.0, 0.0, 0.5], 0.5, [1, 3, 5])
    assert got == (1 if more else 2)


@pytest.mark.parametrize("seed", range(12))
def test_the_third_draft_next_to_its_border(lib, seed):
    """Two rejections with q: W = max(p - (1 + Z) q, 0) and its sum, in exact arithmetic, on both sides of the third test's
    border.  Products of 24-bit factors lose half of their bits where their errors are not kept."""
    g = torch.Generator().manual_seed(seed)
    vocab = 331
    p, q = (torch.softmax(2 * torch.randn(vocab, generator=g), 0) for _ in range(2))
    x1, x2, t0, t1 = torch.randperm(vocab, generator=g)[:4].tolist()
    p[x1] = p[x2] = 0.0
    q[t0] = q[t1] = 0.0
    p[t0], p[t1] = 2.0 ** -20, 1.5 * 2.0 ** -22
    # a token whose third test is open: 0 < W < q Z
    w = (p.double() - q.double()).clamp(min=0)
    w = (p.double() - (1 + w.sum()) * q.double()).clamp(min=0)
    share = w / (q.double() * w.sum())
    x = int(torch.nonzero((share > 0.2) & (share < 0.9))[0])
    assert x not in (x1, x2, t0, t1)
    P, Q = [Fraction(v) for v in p.tolist()], [Fraction(v) for v in q.tolist()]

    def sides(t, u):
        P[t1] = Fraction(t)
        w = [max(a - b, 0) for a, b in zip(P, Q)]
        z = sum(w)
        w = [max(a - (1 + z) * b, 0) for a, b in zip(P, Q)]
        return Fraction(u) * Q[x] * sum(w), w[x], z

    bar, w, z = sides(1.5 * 2.0 ** -22, 1.0)
    assert w > 0 and bar > w
    u = torch.tensor(float(w / bar), dtype=F32).item()
    sign = lambda t: (lambda s: s[0] < s[1])(sides(t, u))  # noqa: E731
    # W(x) and its sum move with the weight of t1: the border, by halving
    grid = [(1 << 23) + i for i in (0, (1 << 23) - 1)]
    lo, hi = grid
    assert sign(lo * 2.0 ** -45) != sign(hi * 2.0 ** -45)
    while hi - lo > 1:
        mid = (lo + hi) // 2
        if sign(mid * 2.0 ** -45) == sign(lo * 2.0 ** -45):
            lo = mid
        else:
            hi = mid
    tested = 0
    for at in (lo, hi):
        for away in (32, 128, 1024, 1 << 14):
            m = at - away if at == lo else at + away
            if not grid[0] <= m <= grid[1]:
                continue
            bar, w, z = sides(m * 2.0 ** -45, u)
            # magnitudes behind either side: u q Z of sums up to 1 + (1 + Z), and p + (1 + Z) q
            size = Fraction(u) * Q[x] * (2 + z) + P[x] + 2 * (1 + z) * Q[x]
            if abs(bar - w) < 2 * bound(vocab) * size:
                continue
            rows = torch.stack([p] * 4)
            rows[:, t1] = m * 2.0 ** -45
            got, _ = call(lib, rows.cuda(), torch.stack([q] * 4).cuda(), [0, x1, x2, x], [0.0, 0.5, 0.5, u], 0.5, [1, 3, 5, 9])
            assert got == (2 if bar < w else 1), (float(bar - w), float(size))
            tested += 1
    assert tested >= 4
