"""What the serving operators around the recurrence are measured on.

The attention layers that stand between KDA layers keep their keys and values
in a paged cache of 4-bit blocks: ``append`` cases write a step's tokens into
it, ``attend`` cases run a decode or speculative step over it.  ``head_norm``
is the gated norm behind the recurrence, ``block_norm`` the norms, gate and
scaled residual between two blocks.

``own`` false: the plain form in elementary torch operations.  True: the calls
of the library.
"""
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
WORKSPACE_BYTES = 20 << 20  # what a program hands to kda_kv4_attend, whatever the sizes
ACT = {"none": 0, "sigmoid": 1, "silu": 2}
_lib = None


def lib():
    """The library's handle, opened once by a program."""
    global _lib
    if _lib is None:
        import kda_linear_attention_gated_gb300 as kda
        _lib = kda.KdaLibrary(torch.float32)
    return _lib


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _append(name, n, t, ragged, hkv, dim, page, dtype, rot, inter, ctx):
    return dict(name=name, op="append", n=n, t=t, ragged=ragged, hkv=hkv, dim=dim, page=page, dtype=dtype, rot=rot,
                inter=inter, ctx=ctx)


def _attend(name, n, t, ragged, ctx, hq, hkv, dim, page, dtype, rot, inter, window):
    return dict(name=name, op="attend", n=n, t=t, ragged=ragged, ctx=ctx, hq=hq, hkv=hkv, dim=dim, page=page,
                dtype=dtype, rot=rot, inter=inter, window=window)


def _head(name, total, heads, dim, src, dtype, act):
    return dict(name=name, op="head_norm", total=total, heads=heads, dim=dim, src=src, dtype=dtype, act=act)


def _block(name, total, hidden, dtype, res, post, act, pre):
    return dict(name=name, op="block_norm", total=total, hidden=hidden, dtype=dtype, res=res, post=post, act=act, pre=pre)


def listed():
    return [
        # one decode token of each of 64 requests
        _append("append_64x1", 64, 1, False, 2, 128, 128, "bf16", 128, False, 4000),
        # a prefill step: eight prompts of 1024 tokens
        _append("append_8x1024", 8, 1024, False, 8, 128, 128, "bf16", 128, False, 0),
        # ragged prompt pieces behind contexts of odd lengths, half the channels rotated as neighbouring pairs, padding
        _append("append_ragged", 13, 301, True, 5, 64, 16, "fp16", 32, True, 777),
        # one request with a short context: latency
        _attend("attend_1x300", 1, 1, False, 300, 12, 2, 128, 128, "bf16", 128, False, 0),
        # a batch of decode tokens behind long contexts: the largest
        _attend("attend_64x8192", 64, 1, False, 8192, 32, 8, 128, 128, "bf16", 128, False, 0),
        # speculative verify: eight tokens a request, ragged contexts, a wide head group
        _attend("attend_verify_32x8", 32, 8, True, 16383, 48, 8, 128, 64, "bf16", 128, False, 0),
        # one very long context, split over the whole card; small heads
        _attend("attend_1x131071", 1, 1, False, 131071, 16, 4, 64, 64, "fp16", 64, True, 0),
        # the output norm behind a decode step (the recurrence's fp32 outputs)
        _head("head_norm_64", 64, 12, 128, "fp32", "bf16", "sigmoid"),
        # the same behind a prefill
        _head("head_norm_8192", 8192, 12, 128, "fp32", "bf16", "sigmoid"),
        # between two blocks of a decode step
        _block("block_norm_64", 64, 4096, "bf16", "bf16", True, "sigmoid", True),
        # between two blocks of a prefill
        _block("block_norm_8192", 8192, 4096, "bf16", "fp32", True, "sigmoid", True),
        # an odd width, fp32 throughout
        _block("block_norm_odd", 1021, 2049, "fp32", "fp32", True, "none", True),
    ]


def _log(rng, lo, hi):
    """A whole number, spread over the logarithm of its range."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["append", "attend", "head_norm", "block_norm"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op in ("append", "attend"):
        dim = rng.choice([64, 128])
        rot = rng.choice([0, dim // 2, dim])
        hkv = rng.randint(1, 8)
        page = 16 * rng.randint(1, 8)
        inter = rng.random() < 0.5
        if op == "append":
            n = _log(rng, 1, 64)
            t = _log(rng, 1, max(1, 8192 // n))
            return {k: v for k, v in _append("", n, t, rng.random() < 0.5, hkv, dim, page, dtype, rot, inter,
                                             rng.randint(0, 5000)).items() if k != "name"}
        n = _log(rng, 1, 64)
        t = _log(rng, 1, 8)
        ctx = _log(rng, 16, min(131071, 400_000 // (n * t)))
        window = rng.choice([0, 0, _log(rng, 1, ctx)])
        return {k: v for k, v in _attend("", n, t, rng.random() < 0.5, ctx, hkv * rng.randint(1, 8), hkv, dim, page,
                                         dtype, rot, inter, window).items() if k != "name"}
    act = rng.choice(["none", "sigmoid", "silu"])
    total = _log(rng, 1, 8192)
    if op == "head_norm":
        src = rng.choice(["fp32", dtype])
        return {k: v for k, v in _head("", total, rng.randint(1, 16), rng.choice([16, 48, 64, 80, 128, 256]), src, dtype,
                                       act).items() if k != "name"}
    res = rng.choice(["fp32", dtype])
    hidden = _log(rng, 64, 8192)
    if rng.random() < 0.5:
        hidden = hidden // 64 * 64
    return {k: v for k, v in _block("", min(total, max(1, (8192 * 4096) // hidden)), hidden, dtype, res,
                                    rng.random() < 0.7, act, rng.random() < 0.8).items() if k != "name"}


# ---------------------------------------------------------------------------
# Lengths: from the case alone
# ---------------------------------------------------------------------------
def lengths(case):
    """(tokens, context before them) of each request.  Ragged: odd lengths of all sizes, the last of four or more a padding request."""
    n, t, ctx = case["n"], case["t"], case["ctx"]
    if not case["ragged"]:
        return [t] * n, [ctx] * n
    rng = random.Random("%s %d %d %d" % (case["op"], n, t, ctx))
    ts = [t] + [rng.randint(1, t) for _ in range(n - 1)]
    cs = [ctx] + [_log(rng, 1, max(1, ctx)) - 1 for _ in range(n - 1)]
    if n >= 4:
        cs[-1] = -ts[-1]
    return ts, cs


def work(case):
    es = {"bf16": 2, "fp16": 2, "fp32": 4}
    e = es[case["dtype"]]
    if case["op"] in ("append", "attend"):
        ts, cs = lengths(case)
        dim, hkv = case["dim"], case["hkv"]
        live = sum(min(t, max(0, t + c)) for t, c in zip(ts, cs))
        if case["op"] == "append":
            # k, v read; the blocks and the values that they stand for written; a table row for each position
            elems = 2 * live * hkv * dim
            rows = {c + j for t, c in zip(ts, cs) for j in range(t) if c + j >= 0}
            out = 2 if case["dtype"] == "fp32" else e
            return {"bytes": elems * (e + 9 / 16 + out) + len(rows) * case["rot"] * 4, "flops": 3.0 * elems}
        w = case["window"] or 1 << 60
        keys = pairs = 0
        for t, c in zip(ts, cs):
            if t + c <= 0:
                continue
            first = max(0, max(0, c) - w + 1)
            keys += t + c - first
            pairs += sum(min(w, c + j + 1) for j in range(t) if c + j >= 0)
        return {"bytes": keys * hkv * dim * 2 * 9 / 16 + 2 * live * case["hq"] * dim * e,
                "flops": 4.0 * pairs * case["hq"] * dim}
    if case["op"] == "head_norm":
        elems = case["total"] * case["heads"] * case["dim"]
        gate = e if case["act"] != "none" else 0
        return {"bytes": elems * (es[case["src"]] + gate + e), "flops": 6.0 * elems}
    elems = case["total"] * case["hidden"]
    gate = e if case["act"] != "none" else 0
    per = e + gate + 2 * es[case["res"]] + (e if case["pre"] else 0)
    return {"bytes": elems * per, "flops": 10.0 * elems}


# ---------------------------------------------------------------------------
# The 4-bit blocks: a value is code x scale, codes e2m1, one e4m3 scale for 16
# neighbouring channels of a token's head.  Sixteen tokens of a head make a
# block of 18 * dim bytes: key codes [16][dim/2]; value codes, in the order in
# which a warp's tensor-core fragments take them; key scales [16][dim/16];
# value scales in fragment order.
# ---------------------------------------------------------------------------
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _encode(x):
    """(codes, e4m3 scale bytes) of x [..., dim] in 32 bits; ties to even.  A group with a value that is not finite: scale NaN, codes 0."""
    g = x.unflatten(-1, (-1, 16))
    amax = g.abs().amax(-1, keepdim=True)
    # divisions, not products with a reciprocal: quotients that lie on a border between two codes stay there
    s8 = (amax / torch.full_like(amax, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()
    y = torch.where(s > 0, g / s, torch.copysign(torch.zeros_like(g), g))
    a = y.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c = c.to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)
    ok = torch.isfinite(amax)
    c = torch.where(ok, c, torch.zeros_like(c))
    b = torch.where(ok, s8.view(torch.uint8), torch.full_like(c[..., :1], 0x7F))
    return c.flatten(-2), b.squeeze(-1)


def _values(codes, scales):
    """The values that codes [..., dim] and scale bytes [..., dim/16] stand for, in 32 bits."""
    lut = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float32, device=codes.device)
    v = lut[codes.int()].unflatten(-1, (-1, 16))
    return (v * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _places(dim, device):
    """Byte places in a block, by token of the block: key codes, value codes [16, dim/2], key scales, value scales [16, dim/16]."""
    cb, ng = dim // 16, dim // 16
    key = torch.arange(16, device=device).view(16, 1)
    half, tq, j = key // 8, key % 8 // 2, key % 2
    byte = torch.arange(dim // 2, device=device).view(1, -1)
    grp = torch.arange(ng, device=device).view(1, -1)
    kc = key * (dim // 2) + byte
    g, b = byte // cb, byte % cb
    vc = 8 * dim + half * (64 * cb) + (g * 4 + tq) * (2 * cb) + j * cb + b
    ks = 16 * dim + key * ng + grp
    vs = 17 * dim + (grp * 4 + tq) * 4 + half * 2 + j
    return kc, vc, ks, vs


def _rotate(x, cos, sin, rot, inter):
    """x [tokens, heads, dim] rotated by table rows [tokens, rot/2]."""
    if rot == 0:
        return x
    c, s = cos.unsqueeze(1), sin.unsqueeze(1)
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        r = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _store(pages, table, req, pos, k, v, page):
    """Writes rows k, v [tokens, hkv, dim] in 32 bits at their positions; returns the values that the cache then stands for."""
    dim = k.shape[-1]
    kc, ks = _encode(k)
    vc, vs = _encode(v)
    live = (pos >= 0).view(-1, 1, 1)
    at = pos.clamp(min=0)
    pid = table[req, at // page].long()
    flat = pages.view(pages.shape[0], pages.shape[1], -1, 18 * dim)
    sel = pos >= 0
    pid, blk, off = pid[sel], (at % page // 16)[sel], (at % 16)[sel]
    heads = torch.arange(k.shape[1], device=k.device)
    places = _places(dim, k.device)
    for data, place in zip((kc[..., 0::2] | (kc[..., 1::2] << 4), vc[..., 0::2] | (vc[..., 1::2] << 4), ks, vs), places):
        p = place[off]
        flat[pid.view(-1, 1, 1), heads.view(1, -1, 1), blk.view(-1, 1, 1), p.unsqueeze(1)] = data[sel]
    zero = torch.zeros((), device=k.device)
    return torch.where(live, _values(kc, ks), zero), torch.where(live, _values(vc, vs), zero)


def _tables(rows, rot, device):
    """cos and sin of position x frequency, the angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / max(rot, 1))
    a = torch.arange(rows, dtype=torch.float64, device=device).view(-1, 1) * f
    return a.cos().float(), a.sin().float()


# ---------------------------------------------------------------------------
# States
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ragged_index(ts, cs):
    cu = [0]
    for t in ts:
        cu.append(cu[-1] + t)
    req = [r for r, t in enumerate(ts) for _ in range(t)]
    pos = [c + j for t, c in zip(ts, cs) for j in range(t)]
    as_t = lambda v, d: torch.tensor(v, dtype=d, device="cuda")  # noqa: E731
    return as_t(cu, torch.int32), as_t(cs, torch.int32), as_t(req, torch.int64), as_t(pos, torch.int64)


def prepare(case, seed):
    g = _gen(seed)
    dt = DT[case["dtype"]]
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"] == "head_norm":
        shape = (case["total"], case["heads"], case["dim"])
        # outputs of the recurrence are small: o = S^T q / sqrt(K)
        s["o"] = (_randn(g, *shape) * 0.1).to(DT[case["src"]])
        s["gate"] = None if case["act"] == "none" else (_randn(g, *shape) * 1.5).to(dt)
        s["weight"] = 1 + 0.1 * _randn(g, case["dim"])
        s["y"] = torch.empty(shape, dtype=dt, device="cuda")
        return s
    if case["op"] == "block_norm":
        shape = (case["total"], case["hidden"])
        s["y"] = (_randn(g, *shape) * 0.5).to(dt)
        s["residual"] = (_randn(g, *shape) * 2).to(DT[case["res"]])
        s["gate"] = None if case["act"] == "none" else (_randn(g, *shape) * 1.5).to(dt)
        s["w_post"] = 1 + 0.1 * _randn(g, case["hidden"]) if case["post"] else None
        s["w_pre"] = 1 + 0.1 * _randn(g, case["hidden"]) if case["pre"] else None
        s["scale"] = 0.5 + 0.1 * _randn(g, case["hidden"])
        s["residual_out"] = torch.empty_like(s["residual"])
        s["x"] = torch.empty(shape, dtype=dt, device="cuda") if case["pre"] else None
        return s
    ts, cs = lengths(case)
    page, dim, hkv, rot = case["page"], case["dim"], case["hkv"], case["rot"]
    ends = [max(0, t + c) for t, c in zip(ts, cs)]
    cols = max(1, -(-max(ends) // page))
    need = sum(-(-e // page) for e in ends)
    num = need + 3
    perm = torch.randperm(num, generator=g, device="cuda").int()
    table = torch.zeros(case["n"], cols, dtype=torch.int32, device="cuda")
    at = 0
    for r, e in enumerate(ends):
        c = -(-e // page)
        table[r, :c] = perm[at:at + c]
        at += c
    s["pages"] = torch.zeros(num, hkv, page // 16, 18 * dim, dtype=torch.uint8, device="cuda")
    s["table"] = table
    s["cu"], s["ctx"], s["req"], s["pos"] = _ragged_index(ts, cs)
    total, s["max_t"], s["max_kv"] = sum(ts), max(ts), max(ends)
    s["cos"], s["sin"] = _tables(max(1, max(ends)), rot, "cuda") if rot else (None, None)
    if case["op"] == "append":
        s["k"] = _randn(g, total, hkv, dim).to(dt)
        s["v"] = _randn(g, total, hkv, dim).to(dt)
        out = torch.bfloat16 if case["dtype"] == "fp32" else dt  # six significant bits: 16-bit values hold them whole
        s["k_out"] = torch.empty(total, hkv, dim, dtype=out, device="cuda")
        s["v_out"] = torch.empty(total, hkv, dim, dtype=out, device="cuda")
        return s
    # a cache as the steps before left it: some key channels larger than others, as in trained models
    gain = torch.exp(0.5 * _randn(g, 1, hkv, dim))
    for r, e in enumerate(ends):
        for a in range(0, e, 16384):
            b = min(e, a + 16384)
            pos = torch.arange(a, b, device="cuda")
            req = torch.full_like(pos, r)
            _store(s["pages"], table, req, pos, _randn(g, b - a, hkv, dim) * gain, _randn(g, b - a, hkv, dim), page)
    s["q"] = (_randn(g, total, case["hq"], dim) * 1.5).to(dt)
    s["o"] = torch.empty_like(s["q"])
    s["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _act(x, act):
    return x if act == "none" else torch.sigmoid(x) if act == "sigmoid" else x * torch.sigmoid(x)


def _rms(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


def _plain_head_norm(s):
    y = _rms(s["o"].float()) * s["weight"]
    if s["gate"] is not None:
        y = y * _act(s["gate"].float(), s["case"]["act"])
    return {"y": y.to(s["y"].dtype)}


def _plain_block_norm(s):
    z = s["y"].float()
    if s["w_post"] is not None:
        z = _rms(z) * s["w_post"]
    z = z * s["scale"]
    if s["gate"] is not None:
        z = z * _act(s["gate"].float(), s["case"]["act"])
    h = 0.9 * s["residual"].float() + 0.7 * z
    out = {"residual": h.to(s["residual"].dtype)}
    if s["w_pre"] is not None:
        out["x"] = (_rms(h) * s["w_pre"]).to(s["x"].dtype)
    return out


def _row_tables(s):
    at = s["pos"].clamp(min=0)
    return (s["cos"][at], s["sin"][at]) if s["cos"] is not None else (None, None)


def _plain_append(s):
    c = s["case"]
    cos, sin = _row_tables(s)
    k = _rotate(s["k"].float(), cos, sin, c["rot"], c["inter"])
    kq, vq = _store(s["pages"], s["table"], s["req"], s["pos"], k, s["v"].float(), c["page"])
    return {"pages": s["pages"], "k": kq.to(s["k_out"].dtype), "v": vq.to(s["v_out"].dtype)}


def _plain_attend(s):
    c = s["case"]
    n, hq, hkv, dim, page, t = c["n"], c["hq"], c["hkv"], c["dim"], c["page"], s["max_t"]
    grp = hq // hkv
    cos, sin = _row_tables(s)
    q = _rotate(s["q"].float(), cos, sin, c["rot"], c["inter"])
    qp = q.new_zeros(n, t, hq, dim)
    j = torch.arange(q.shape[0], device=q.device) - s["cu"][:-1].long()[s["req"]]
    qp[s["req"], j] = q
    qp = qp.view(n, t, hkv, grp, dim).permute(0, 2, 1, 3, 4).reshape(n, hkv, t * grp, dim)
    cols = max(1, -(-s["max_kv"] // page))
    blocks = s["pages"][s["table"][:, :cols].long()].transpose(1, 2).reshape(n, hkv, -1, 18 * dim)
    kc, vc, ks, vs = _places(dim, q.device)
    lut = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float32, device=q.device)
    byte = torch.arange(256, device=q.device)
    pair = torch.stack((lut[byte & 15], lut[byte >> 4]), -1)

    def rows(codes, scales):
        v = pair[blocks[..., codes].int()].flatten(-2).unflatten(-1, (-1, 16))
        v = v * blocks[..., scales].view(torch.float8_e4m3fn).float().unsqueeze(-1)
        return v.flatten(-2).flatten(2, 3)

    pos = torch.full((n, t), -1, dtype=torch.int64, device=q.device)
    pos[s["req"], j] = s["pos"]
    keys = torch.arange(blocks.shape[2] * 16, device=q.device)
    seen = keys.view(1, 1, -1) <= pos.unsqueeze(-1)
    if c["window"]:
        seen = seen & (keys.view(1, 1, -1) > pos.unsqueeze(-1) - c["window"])
    seen = seen.unsqueeze(2).expand(n, t, grp, -1).reshape(n, 1, t * grp, -1)
    score = torch.matmul(qp, rows(kc, ks).transpose(-1, -2)) * dim ** -0.5
    score = score.masked_fill(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    o = torch.matmul(p, rows(vc, vs)) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(n, hkv, t, grp, dim).permute(0, 2, 1, 3, 4).reshape(n, t, hq, dim)
    return {"o": o[s["req"], j].to(s["o"].dtype)}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "head_norm": _plain_head_norm,
                "block_norm": _plain_block_norm}[c["op"]](s)
    L = lib()
    if c["op"] == "append":
        L.kda_kv4_append(s["pages"], s["table"], s["ctx"], s["k"], s["v"], s["status"], cu_seqlens=s["cu"],
                         max_t=s["max_t"], cos=s["cos"], sin=s["sin"], interleaved=c["inter"], k_out=s["k_out"],
                         v_out=s["v_out"])
        return {"pages": s["pages"], "k": s["k_out"], "v": s["v_out"]}
    if c["op"] == "attend":
        L.kda_kv4_attend(s["pages"], s["table"], s["ctx"], s["q"], s["o"], s["workspace"], s["status"],
                         cu_seqlens=s["cu"], max_t=s["max_t"], cos=s["cos"], sin=s["sin"], interleaved=c["inter"],
                         window=c["window"])
        return {"o": s["o"]}
    if c["op"] == "head_norm":
        L.kda_head_norm(s["o"], s["weight"], s["y"], gate=s["gate"], activation=ACT[c["act"]])
        return {"y": s["y"]}
    L.kda_block_norm(s["residual"], s["y"], s["residual_out"], w_post=s["w_post"], gate=s["gate"],
                     activation=ACT[c["act"]], scale=s["scale"], w_pre=s["w_pre"], x=s["x"], residual_scale=0.9,
                     branch_scale=0.7)
    out = {"residual": s["residual_out"]}
    if s["x"] is not None:
        out["x"] = s["x"]
    return out


# ---------------------------------------------------------------------------
# The definitions in 64 bits, request by request
# ---------------------------------------------------------------------------
def _exact_rotate(x, pos, rot, inter):
    """x [tokens, heads, dim] at positions pos, in 64 bits."""
    if rot == 0:
        return x
    i = torch.arange(rot // 2, device=x.device)
    # the tables are inputs in 32 bits
    a = pos.double().view(-1, 1) * (10000.0 ** (-2.0 * i.double() / rot)).view(1, -1)
    c, s = a.cos().float().double().unsqueeze(1), a.sin().float().double().unsqueeze(1)
    first, second = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    y = x.clone()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


def _exact_round(x):
    """x [..., dim] in 64 bits to the nearest values that a group's scale and codes can hold."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    a = g.abs().amax(-1, keepdim=True) / 6
    steps = torch.tensor([2.0 ** (i - 9) for i in range(18)], dtype=torch.float64, device=x.device)  # exact powers
    step = steps[(torch.frexp(a).exponent + 5).clamp(0, 17).long()]  # a in [2^-6, 2^-5): 2^-9, and below
    sc = torch.clamp(torch.round(a / step) * step, max=448.0)
    y = torch.where(sc > 0, g / torch.where(sc > 0, sc, torch.ones_like(sc)), torch.zeros_like(g))
    # codes lie 1/2 apart below 2, 1 apart below 4, 2 apart above; round() takes ties to the even one
    m = y.abs()
    m = torch.where(m < 2, torch.round(2 * m) / 2, torch.where(m < 4, torch.round(m), (2 * torch.round(m / 2)).clamp(max=6)))
    return (torch.sign(y) * m * sc).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "head_norm":
        o = s["o"].double()
        y = o / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-6) * s["weight"].double()
        if s["gate"] is not None:
            z = s["gate"].double()
            y = y / (1 + torch.exp(-z)) * (z if case["act"] == "silu" else 1)
        return {"y": y}
    if case["op"] == "block_norm":
        z = s["y"].double()
        if case["post"]:
            z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + 1e-6) * s["w_post"].double()
        if s["gate"] is not None:
            a = s["gate"].double()
            z = z / (1 + torch.exp(-a)) * (a if case["act"] == "silu" else 1)
        h = 0.9 * s["residual"].double() + 0.7 * s["scale"].double() * z
        out = {"residual": h}
        if case["pre"]:
            out["x"] = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * s["w_pre"].double()
        return out
    if case["op"] == "append":
        live = (s["pos"] >= 0).view(-1, 1, 1)
        k = _exact_round(_exact_rotate(s["k"].double(), s["pos"], case["rot"], case["inter"]))
        v = _exact_round(s["v"].double())
        return {"pages": None, "k": torch.where(live, k, 0.0), "v": torch.where(live, v, 0.0)}
    ts, cs = lengths(case)
    hkv, dim, page, grp = case["hkv"], case["dim"], case["page"], case["hq"] // case["hkv"]
    q = _exact_rotate(s["q"].double(), s["pos"], case["rot"], case["inter"])
    o, at = torch.zeros_like(q), 0
    grid = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
    for r, (t, ctx) in enumerate(zip(ts, cs)):
        end = max(0, t + ctx)
        for h in range(hkv if end else 0):
            b = s["pages"][s["table"][r, : -(-end // page)].long(), h].reshape(-1, 18 * dim)
            codes_k = b[:, : 8 * dim].reshape(-1, 16, dim // 2)
            # value codes: [half][channel eighth][quad][token of a pair][bytes] of each block
            codes_v = b[:, 8 * dim: 16 * dim].reshape(-1, 2, 8, 4, 2, dim // 16).permute(0, 1, 3, 4, 2, 5)
            codes_v = codes_v.reshape(-1, 16, dim // 2)
            sk = b[:, 16 * dim: 17 * dim].reshape(-1, 16, dim // 16)
            sv = b[:, 17 * dim:].reshape(-1, dim // 16, 4, 2, 2).permute(0, 3, 2, 4, 1).reshape(-1, 16, dim // 16)

            def rows(codes, scales):
                c = torch.stack((codes & 15, codes >> 4), -1).reshape(-1, dim)[:end].long()
                w = scales.contiguous().view(torch.float8_e4m3fn).double().reshape(-1, dim // 16)[:end]
                return torch.where(c >= 8, -grid[c & 7], grid[c & 7]) * w.repeat_interleave(16, -1)

            k, v = rows(codes_k, sk), rows(codes_v, sv)
            x = q[at:at + t, h * grp:(h + 1) * grp]
            w = torch.einsum("tgd,pd->tgp", x, k) / dim ** 0.5
            p = torch.arange(end, device="cuda").view(1, 1, -1)
            mine = (ctx + torch.arange(t, device="cuda")).view(-1, 1, 1)
            out = p > mine
            if case["window"]:
                out = out | (p <= mine - case["window"])
            w = torch.softmax(w.masked_fill(out, float("-inf")), -1).nan_to_num(0.0)
            o[at:at + t, h * grp:(h + 1) * grp] = torch.einsum("tgp,pd->tgd", w, v)
        at += t
    return {"o": o}
