"""Masks that are no tree's (an ancestor's ancestors missing, any bits at all): what the kernels do with them, restated, ends,
takes every token once and stays within the request.  (No GPU: such masks are the caller's mistake, and their results are
anything.)"""
import random

import pytest


def masks(t, kind, seed):
    rng = random.Random(f"{t} {kind} {seed}")
    if kind == "random":
        return [rng.getrandbits(64) for _ in range(t)]
    if kind == "sparse":
        return [sum(1 << rng.randrange(64) for _ in range(rng.randrange(4))) for _ in range(t)]
    if kind == "parents only":
        return [1 << rng.randrange(i) if i else 0 for i in range(t)]
    return [{"ones": (1 << 64) - 1, "zeros": 0, "even": 0x5555555555555555}[kind]] * t


def above(tree, j):
    """The ancestors that the kernels see: the bits below a token's own."""
    return tree[j] & ((1 << j) - 1)


def top(m):
    return m.bit_length() - 1


def low(m):
    return (m & -m).bit_length() - 1


KINDS = ["random", "sparse", "parents only", "ones", "zeros", "even"]


@pytest.mark.parametrize("t", [1, 2, 7, 33, 64])
@pytest.mark.parametrize("kind", KINDS)
def test_depth_first_order(t, kind):
    """kda_step_tree: leaves two at a time, then an inner child in place; another branch from the lowest token left."""
    for seed in range(20):
        tree = masks(t, kind, seed)
        up = [above(tree, j) for j in range(t)]
        child = [0] * t
        for j in range(t):
            if up[j]:
                child[top(up[j])] |= 1 << j
        todo = (1 << t) - 1
        leaves = sum(1 << j for j in range(t) if not child[j])
        kids = sum(1 << j for j in range(t) if not up[j])
        taken, rounds = [], 0
        while todo:
            rounds += 1
            assert rounds <= t
            kids &= todo
            if not kids:
                j = low(todo)
                m = up[j]
                while m:            # replayed: tokens that are done
                    assert low(m) in taken
                    m &= m - 1
                kids = child[top(up[j])] & todo if up[j] else 1 << j
            ends, inner = kids & leaves, kids & ~leaves
            left = ends & (ends - 1)
            down = not ends or (not left and inner)
            js = [low(ends if ends else inner)]
            if left:
                js.append(low(left))
            elif inner and ends:
                js.append(low(inner))
            assert all(0 <= j < t and todo >> j & 1 for j in js) and len(set(js)) == len(js)
            taken += js
            for j in js:
                todo &= ~(1 << j)
            if down:
                kids = child[js[-1]]
        assert sorted(taken) == list(range(t))


@pytest.mark.parametrize("t", [1, 5, 64])
@pytest.mark.parametrize("kind", KINDS)
def test_taps_of_the_convolution(t, kind):
    """kda_conv_step_tree: rows of history and tokens, for every width."""
    for seed in range(10):
        tree = masks(t, kind, seed)
        for kw in range(1, 9):
            for j in range(t):
                m, hist = above(tree, j) | 1 << j, kw - 2
                for _ in range(kw):
                    row = hist
                    if m:
                        row = kw - 1 + top(m)
                        m ^= 1 << top(m)
                    else:
                        hist -= 1
                    assert 0 <= row < kw - 1 + t


@pytest.mark.parametrize("t", [1, 6, 64])
@pytest.mark.parametrize("kind", KINDS)
def test_walk_of_the_acceptance(t, kind):
    """kda_accept, whatever is accepted: children lie behind their parent, so that the path is no longer than the request."""
    for seed in range(10):
        tree, rng = masks(t, kind, seed), random.Random(seed)
        child = [0] * t
        for j in range(t):
            if above(tree, j):
                child[top(above(tree, j))] |= 1 << j
        for odds in (0.0, 0.5, 1.0):
            path, rest = [0], child[0]
            while rest:
                i = low(rest)
                rest &= rest - 1
                if rng.random() < odds:
                    assert path[-1] < i < t
                    path.append(i)
                    rest = child[i]
            assert len(path) <= t


@pytest.mark.parametrize("t", [1, 6, 64])
@pytest.mark.parametrize("kind", KINDS)
def test_positions_of_the_attention(t, kind):
    """kda_kv4_append_tree and kda_kv4_attend_tree: depths stay within the rotation's rows (up to ctx + t - 1), keys within
    the request's, and a window leaves the token itself."""
    for seed in range(10):
        tree = masks(t, kind, seed)
        for j in range(t):
            own = above(tree, j) | 1 << j
            depth = bin(own).count("1") - 1
            assert 0 <= depth <= j < t and own < 1 << t
            for window in (1, 3, 64):
                seen = own
                for _ in range(max(0, depth + 1 - window)):
                    seen &= seen - 1
                assert seen >> j == 1 and bin(seen).count("1") == min(depth + 1, window)
