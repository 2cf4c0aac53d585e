"""Plain restatements of the operators around the recurrence, for the tests:
the 4-bit block format with its encoder step by step in fp32 (so that bytes can
be compared for equality), attention and norms in fp64."""
from __future__ import annotations

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def half_step(dtype) -> float:
    """Largest relative error of one rounding to nearest."""
    return torch.finfo(dtype).eps / 2


# -- format -------------------------------------------------------------------
def encode(x):
    """(codes [..., dim], e4m3 bytes [..., dim / 16]) of fp32 x, each step in fp32."""
    assert x.dtype == torch.float32
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    amax = g.abs().amax(-1, keepdim=True)           # NaN if there is one
    fine = torch.isfinite(amax)
    s8 = (amax / torch.full_like(amax, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()
    y = torch.where(s > 0, g / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(g)).abs()
    # to nearest, ties to the even code: borders that belong to the code above are 0.75, 1.75, 3.5
    c = torch.zeros(y.shape, dtype=torch.uint8)
    for border, above in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        c += ((y >= border) if above else (y > border)).to(torch.uint8)
    c += 8 * torch.signbit(g).to(torch.uint8)
    c = torch.where(fine, c, torch.zeros_like(c))
    b = torch.where(fine, s8.view(torch.uint8), torch.full(fine.shape, 0x7F, dtype=torch.uint8))
    return c.flatten(-2), b.squeeze(-1)


def decode(codes, scales):
    """fp64 values of codes and scale bytes."""
    v = torch.where(codes >= 8, -1.0, 1.0).double() * E2M1[(codes & 7).long()]
    return v * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


def pack(codes_k, scales_k, codes_v, scales_v):
    """Blocks [heads, blocks, 18 dim] of [tokens, heads, ...], tokens a multiple of 16; byte by byte from the header's layout."""
    t, h, dim = codes_k.shape
    c = dim // 16
    out = torch.zeros(h, t // 16, 18 * dim, dtype=torch.uint8)
    two = lambda x: x[..., 0::2] | (x[..., 1::2] << 4)  # noqa: E731
    kb, vb = two(codes_k), two(codes_v)
    for w in range(16):
        sl = slice(w, None, 16)
        out[:, :, w * dim // 2:(w + 1) * dim // 2] = kb[sl].transpose(0, 1)
        out[:, :, 16 * dim + w * c:16 * dim + (w + 1) * c] = scales_k[sl].transpose(0, 1)
        for j in range(dim // 2):
            at = w // 8 * 64 * c + (j // c * 4 + w % 8 // 2) * 2 * c + w % 2 * c + j % c
            out[:, :, 8 * dim + at] = vb[sl, :, j].transpose(0, 1)
        for i in range(c):
            out[:, :, 17 * dim + (i * 4 + w % 8 // 2) * 4 + w // 8 * 2 + w % 2] = scales_v[sl, :, i].transpose(0, 1)
    return out


def rotate32(x, cos, sin, interleaved):
    """fp32 x [tokens, heads, dim] rotated by rows cos, sin [tokens, rot / 2], every product and sum rounded once."""
    half = cos.shape[1]
    c, s = cos[:, None], sin[:, None]
    y = x.clone()
    ia = torch.arange(half) * 2 if interleaved else torch.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def tables(rows, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


class Cache:
    """A paged cache on the CPU: the values of every request's positions, and the packed pages."""

    def __init__(self, ends, heads, dim, page, gen, spare=2, v_gain=1.0, poison=None):
        self.heads, self.dim, self.page = heads, dim, page
        cols = max(1, max(-(-e // page) for e in ends))
        need = sum(-(-e // page) for e in ends) + spare
        perm = torch.randperm(need, generator=gen).int()
        self.table = torch.full((len(ends), cols), -7, dtype=torch.int32)
        # never-written places hold bytes that read back as NaN
        self.pages = torch.full((need, heads, page // 16, 18 * dim), 0x7F, dtype=torch.uint8)
        self.k, self.v, at = [], [], 0
        for r, e in enumerate(ends):
            n = -(-e // page)
            self.table[r, :n] = perm[at:at + n]
            at += n
            full = n * page
            ck, sk = encode(torch.randn(full, heads, dim, generator=gen))
            cv, sv = encode(torch.randn(full, heads, dim, generator=gen) * v_gain)
            if poison is not None:
                poison(r, sk, sv)
            sk[e:], sv[e:] = 0x7F, 0x7F
            blocks = pack(ck, sk, cv, sv) if n else torch.zeros(heads, 0, 18 * dim, dtype=torch.uint8)
            for i in range(n):
                self.pages[self.table[r, i]] = blocks[:, i * page // 16:(i + 1) * page // 16]
            self.k.append(decode(ck[:e], sk[:e]))
            self.v.append(decode(cv[:e], sv[:e]))


def attend(cache, ctx, lens, q, cos, sin, interleaved, window=0, scale=None, k_scale=1.0, v_scale=1.0):
    """(o, bound) in fp64: o by its definition, and max |v| and the sums that the tolerance is made of."""
    dim, hq = q.shape[-1], q.shape[1]
    grp = hq // cache.heads
    scale = dim ** -0.5 if scale is None else scale
    o = torch.zeros(q.shape, dtype=torch.float64)
    err = torch.zeros(q.shape[:2], dtype=torch.float64)      # per row: largest score error in units of the factor u
    big = torch.zeros(q.shape[:2], dtype=torch.float64)      # per row: largest |value| seen
    top = torch.zeros(q.shape[:2], dtype=torch.float64)      # per row: largest |score|
    at = 0
    for r, t in enumerate(lens):
        for j in range(t):
            p = ctx[r] + j
            if p < 0:
                continue
            first = max(0, p - window + 1) if window else 0
            for h in range(hq):
                x = q[at + j, h].double()
                if cos is not None:
                    x = rotate32(x[None, None], cos[p:p + 1].double(), sin[p:p + 1].double(), interleaved)[0, 0]
                k, v = cache.k[r][first:p + 1, h // grp] * k_scale, cache.v[r][first:p + 1, h // grp] * v_scale
                s = scale * (k @ x)
                w = torch.softmax(s, 0)
                o[at + j, h] = w @ v
                err[at + j, h] = (abs(scale) * (k.abs() @ q[at + j, h].double().abs())).max()
                big[at + j, h] = v.abs().max()
                top[at + j, h] = s.abs().max()
        at += t
    return o, err, big, top


def attend_tolerance(o, err, big, top, dtype, split):
    """Elementwise bound of the kernel's error.  A score is off by at most u
    times the sum of |products| (the query's rounding: 2^-12, or 2^-22 with
    remainders; rotation in fp32: 3 roundings; fp32 sums of up to 17 terms of an
    mma chain) and by the rounding of its own product with the row factor and
    of the difference to the maximum (2 * 2^-24 of |score|); an exponential by
    2^-22, a probability by its rounding.  Numerator and denominator both carry
    it: 2 times, times the largest value.  Sums over keys in fp32: the order of
    a few hundred terms, 2^-17 at most.  Then the output's rounding."""
    u = (2.0 ** -22 if split else 2.0 ** -12) + 20 * 2.0 ** -24
    e = u * err + 2.0 ** -23 * top
    p = 2.0 ** -21 if split else 2.0 ** -12
    return half_step(dtype) * o.abs() + (big * (2 * (torch.expm1(e) + p) + 2.0 ** -17)).unsqueeze(-1)


# -- norms --------------------------------------------------------------------
def act(x, kind):
    return x if kind == 0 else torch.sigmoid(x) if kind == 1 else x * torch.sigmoid(x)


def rms(x, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def head_norm(o, weight, gate, kind, eps):
    y = rms(o.double(), eps) * weight.double()
    return y if gate is None else y * act(gate.double(), kind)


def block_norm(residual, y, w_post, gate, kind, scale, w_pre, a, b, eps):
    h = residual.double()
    if y is not None:
        z = y.double()
        if w_post is not None:
            z = rms(z, eps) * w_post.double()
        if scale is not None:
            z = z * scale.double()
        if gate is not None:
            z = z * act(gate.double(), kind)
        z, h = b * z, a * h
        mag = h.abs() + z.abs()
        h = h + z
    else:
        mag = h.abs()
    x = rms(h, eps)
    if w_pre is not None:
        x = x * w_pre.double()
    return h, mag, x
