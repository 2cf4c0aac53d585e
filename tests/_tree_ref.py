"""Plain restatements in 64 bits of a speculative step over a tree of drafted
tokens, request by request and token by token."""
from __future__ import annotations

import random

import torch

U = 2.0 ** -24      # half a step of fp32


def parents(t, shape, seed=0):
    """Parents of t tokens (-1: the context), which come first."""
    rng = random.Random(f"{t} {shape} {seed}")
    out = []
    for i in range(t):
        if i == 0 or shape == "forest" and rng.random() < 0.3:
            out.append(-1)
        elif shape == "chain":
            out.append(i - 1)
        elif shape == "star":
            out.append(0)
        else:
            out.append(rng.randint(max(0, i - 6), i - 1))
    return out


def ancestors(par):
    """The tokens on each token's path, itself last."""
    paths = []
    for i, p in enumerate(par):
        paths.append((paths[p] if p >= 0 else []) + [i])
    return paths


def masks(pars, device="cuda"):
    """int64 masks of several requests' trees."""
    out = []
    for par in pars:
        for path in ancestors(par):
            m = sum(1 << i for i in path)
            out.append(m - (1 << 64) if m >> 63 else m)
    return torch.tensor(out, dtype=torch.int64, device=device)


def step(S0, par, q, k, v, a, b, a_log=None, dt_bias=None):
    """Outputs [t, hv, V] and states [t, hv, K, V] with elementwise bounds of an fp32 kernel's error.

    Bounds, U half a step: a normalised vector's entry is off by (K + 8) U of itself (the sum of squares, the root, two
    products); a gate by 16 U and, with the learned scale, by 8 U of its exponent as well (the exponential of a
    rounded product); a sum of K products by (K + 2) U of the sum of magnitudes; each product and sum of the update
    by U.  Errors of the parent's state go through with the factors of the update."""
    t, hv, kd = a.shape
    rep = hv // q.shape[1]
    q, k, v, a, b = (x.double() for x in (q, k, v, a, b))
    q, k = (x.repeat_interleave(rep, 1) for x in (q, k))
    qh, kh = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6) for x in (q, k))
    if a_log is None:
        expo = torch.nn.functional.softplus(a)
        e_alpha = torch.full_like(a, 16 * U)
    else:
        expo = torch.exp(a_log.double()).view(hv, 1) * torch.nn.functional.softplus(a + (0 if dt_bias is None else dt_bias.double()))
        e_alpha = (16 + 8 * expo) * U
    alpha, beta = torch.exp(-expo), torch.sigmoid(b)
    n = (kd + 8) * U
    o, eo, states, es = [], [], [], []
    for j in range(t):
        S, e = (states[par[j]], es[par[j]]) if par[j] >= 0 else (S0.double(), torch.zeros_like(S0, dtype=torch.float64))
        al, kj, qj, bt = alpha[j].unsqueeze(-1), kh[j].unsqueeze(-1), qh[j].unsqueeze(-1), beta[j].unsqueeze(-1)
        S = S * al
        e = e * al + S.abs() * (e_alpha[j].unsqueeze(-1) + 2 * U)
        u = (S * kj).sum(-2)
        mag = (S.abs() * kj.abs()).sum(-2)
        eu = (e * kj.abs()).sum(-2) + mag * (n + (kd + 2) * U)
        d = bt * (v[j] - u)
        ed = bt * (eu + 4 * U * (v[j].abs() + mag)) + 8 * U * d.abs()
        new = S + kj * d.unsqueeze(-2)
        e = e + kj.abs() * (ed + (n + 2 * U) * d.abs()).unsqueeze(-2) + U * new.abs()
        out = (new * qj).sum(-2) * kd ** -0.5
        # computed as S^T q + (k . q) d: both sums' errors
        kq = (kj.abs() * qj.abs()).sum(-2)
        eo_j = ((e * qj.abs()).sum(-2) + (S.abs() * qj.abs()).sum(-2) * (n + (kd + 2) * U) + kq * (ed + d.abs() * (2 * n + (kd + 4) * U))) * kd ** -0.5
        o.append(out)
        eo.append(eo_j + 8 * U * out.abs())
        states.append(new)
        es.append(e)
    return (torch.stack(x) for x in (o, eo, states, es))


def conv(hist, par, x, weight, bias, silu):
    """y [t, C] and the bound of an fp32 kernel's error: hist [KW - 1, C] the inputs before the tree."""
    kw = weight.shape[1]
    w = weight.double()
    ys, es = [], []
    for path in ancestors(par):
        z = torch.cat((hist.double(), x[path].double()))[-kw:] if kw > 1 else x[path[-1:]].double()
        y = (z.T * w).sum(-1)
        mag = (z.T * w).abs().sum(-1)
        if bias is not None:
            y, mag = y + bias.double(), mag + bias.double().abs()
        e = (kw + 2) * U * mag
        if silu:
            # |silu'| < 1.1; the exponential's and the quotient's intrinsics: 2 + 1.2 |y| and 2 units of 2 U
            s = y * torch.sigmoid(y)
            e = 1.1 * e + (8 + 3 * y.abs()) * U * s.abs()
            y = s
        ys.append(y)
        es.append(e)
    return torch.stack(ys), torch.stack(es)


def accept(p, q, tokens, par, u, u_last):
    """(path, next token) of one request, in 64 bits; p, q [t, vocab]."""
    p = torch.where(p.double() > 0, p.double(), torch.zeros(()).double())
    q = None if q is None else torch.where(q.double() > 0, q.double(), torch.zeros(()).double())
    vocab, cur, path = p.shape[1], 0, [0]
    w, z = p[0], 1.0
    for i in range(1, len(par)):
        if par[i] != cur:
            continue
        x = int(tokens[i])
        if not 0 <= x < vocab:
            continue
        held, draft = float(w[x]), 1.0 if q is None else float(q[cur, x])
        if float(u[i]) * draft * z < held:
            cur = i
            path.append(i)
            w, z = p[i], 1.0
        elif q is None:
            w = w.clone()
            w[x] = 0.0
            z -= held
        else:
            w = (w - z * q[cur]).clamp(min=0)
            z = float(w.sum())
    if not float(w.sum()) > 0:
        w = p[cur]
    some = torch.nonzero(w > 0).flatten()
    if not some.numel() or not float(w.sum()) < float("inf"):
        return path, -1
    cum = torch.cumsum(w[some], 0)
    over = torch.nonzero(cum > float(u_last) * float(cum[-1])).flatten()
    return path, int(some[over[0]]) if over.numel() else int(some[-1])


def attend(cache, ctx, pars, q, cos, sin, interleaved, window=0, scale=None, k_scale=1.0, v_scale=1.0):
    """As attend of _layer_ref, over trees: (o, err, big, top)."""
    from _layer_ref import rotate32
    dim, hq = q.shape[-1], q.shape[1]
    grp = hq // cache.heads
    scale = dim ** -0.5 if scale is None else scale
    o = torch.zeros(q.shape, dtype=torch.float64)
    err, big, top = (torch.zeros(q.shape[:2], dtype=torch.float64) for _ in range(3))
    at = 0
    for r, par in enumerate(pars):
        for path in ancestors(par):
            depth = len(path) - 1
            pos = ctx[r] + depth
            if ctx[r] >= 0:
                first = max(0, pos - window + 1) if window else 0
                keys = list(range(first, ctx[r])) + [ctx[r] + i for d, i in enumerate(path) if not window or d > depth - window]
                for h in range(hq):
                    x = q[at, h].double()
                    if cos is not None:
                        x = rotate32(x[None, None], cos[pos:pos + 1].double(), sin[pos:pos + 1].double(), interleaved)[0, 0]
                    k, v = cache.k[r][keys, h // grp] * k_scale, cache.v[r][keys, h // grp] * v_scale
                    s = scale * (k @ x)
                    o[at, h] = torch.softmax(s, 0) @ v
                    err[at, h] = (abs(scale) * (k.abs() @ q[at, h].double().abs())).max()
                    big[at, h] = v.abs().max()
                    top[at, h] = s.abs().max()
            at += 1
    return o, err, big, top
