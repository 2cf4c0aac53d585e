"""What the operators of a speculative step over a tree of drafted tokens are
measured on.

A request's drafted tokens form a tree behind its context: ``tree`` holds a
mask for each token, bit i for the i-th token of its request, of the token's
ancestors and itself (a chain of drafts is the tree in which each token's
ancestors are all before it).  ``attend`` cases run a full attention layer over
the tree and the paged 4-bit cache, ``step`` cases the recurrence with a state
for every token, ``conv`` cases the short convolution in front of it, and
``accept`` cases walk the tree: drafts are accepted or rejected against the
target's probabilities with given random numbers, and the next token is drawn.

``own`` false: the plain form in elementary torch operations.  True: the calls
of the library.
"""
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
WORKSPACE_BYTES = 64 << 20  # what a program hands to kda_kv4_attend_tree, whatever the sizes
_lib = {}


def lib(pool_dtype=torch.float32):
    """The library's handle for a pool dtype, opened once by a program."""
    if pool_dtype not in _lib:
        import kda_linear_attention_gated_gb300 as kda
        _lib[pool_dtype] = kda.KdaLibrary(pool_dtype)
    return _lib[pool_dtype]


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _accept(name, n, t, ragged, shape, vocab, dtype, drawn):
    return dict(name=name, op="accept", n=n, t=t, ragged=ragged, shape=shape, vocab=vocab, dtype=dtype, drawn=drawn)


def _attend(name, n, t, ragged, shape, ctx, hq, hkv, dim, page, dtype, rot, inter, window):
    return dict(name=name, op="attend", n=n, t=t, ragged=ragged, shape=shape, ctx=ctx, hq=hq, hkv=hkv, dim=dim,
                page=page, dtype=dtype, rot=rot, inter=inter, window=window)


def _step(name, n, t, ragged, shape, hv, hqk, kd, vd, pool, dtype, learned):
    return dict(name=name, op="step", n=n, t=t, ragged=ragged, shape=shape, hv=hv, hqk=hqk, kd=kd, vd=vd, pool=pool,
                dtype=dtype, learned=learned)


def _conv(name, n, t, ragged, shape, channels, width, dtype, silu, bias):
    return dict(name=name, op="conv", n=n, t=t, ragged=ragged, shape=shape, channels=channels, width=width, dtype=dtype,
                silu=silu, bias=bias)


def listed():
    return [
        # one request's chain of four drafts behind its last token: latency
        _accept("accept_1x5", 1, 5, False, "chain", 32000, "fp32", True),
        # a batch of chains as speculative verify has them, a large vocabulary
        _accept("accept_64x8", 64, 8, False, "chain", 131072, "fp32", True),
        # trees of ragged sizes with several drafts of one token, an odd vocabulary, probabilities in 16 bits
        _accept("accept_ragged", 13, 37, True, "wide", 50021, "bf16", True),
        # one request with a small tree and a short context: latency
        _attend("attend_1x7", 1, 7, False, "wide", 300, 12, 2, 128, 128, "bf16", 128, False, 0),
        # ragged contexts with trees of up to 16 tokens, a wide head group
        _attend("attend_ragged", 32, 16, True, "deep", 16383, 48, 8, 128, 64, "bf16", 128, False, 0),
        # full trees behind long contexts: the largest
        _attend("attend_8x64", 8, 64, False, "wide", 8192, 32, 8, 128, 128, "bf16", 128, False, 0),
        # one very long context with a tree, small heads, fp16
        _attend("attend_1x131071", 1, 24, False, "wide", 131071, 16, 4, 64, 64, "fp16", 64, True, 0),
        # one request's tree in a KDA layer: latency
        _step("step_1x8", 1, 8, False, "wide", 12, 12, 128, 128, "fp32", "bf16", False),
        # full trees on an fp16 pool: 512 states written
        _step("step_16x32", 16, 32, False, "wide", 12, 12, 128, 128, "fp16", "bf16", False),
        # ragged trees on an fp32 pool, grouped heads of odd sizes, the learned gate scale
        _step("step_ragged", 13, 48, True, "deep", 6, 3, 96, 80, "fp32", "fp16", True),
        # the convolution in front of one request's step: latency
        _conv("conv_1x8", 1, 8, False, "wide", 4608, 4, "bf16", True, True),
        # full trees of a batch
        _conv("conv_32x64", 32, 64, False, "wide", 4608, 4, "bf16", True, True),
    ]


def _log(rng, lo, hi):
    """A whole number, spread over the logarithm of its range."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["accept", "attend", "step", "conv"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    shape = rng.choice(["chain", "deep", "wide"])
    ragged = rng.random() < 0.5
    n, t = _log(rng, 1, 64), _log(rng, 1, 64)
    if op == "accept":
        vocab = _log(rng, 1000, 200_000)
        t = max(1, min(t, (64 * 8 * 131072) // (n * vocab)))
        c = _accept("", n, t, ragged, shape, vocab, dtype, rng.random() < 0.6)
    elif op == "attend":
        dim = rng.choice([64, 128])
        hkv = rng.randint(1, 8)
        hq = hkv * rng.randint(1, 8)
        n = min(n, max(1, 2000 // t))
        ctx = _log(rng, 16, max(17, min(131071, 400_000 // n, (8 * 64 * 8192 * 32 // 2) // (n * t * hq))))
        c = _attend("", n, t, ragged, shape, ctx, hq, hkv, dim, 16 * rng.randint(1, 8), dtype,
                    rng.choice([0, dim // 2, dim]), rng.random() < 0.5, rng.choice([0, 0, _log(rng, 1, ctx)]))
    elif op == "step":
        hqk = rng.randint(1, 6)
        hv = hqk * rng.randint(1, 12 // hqk)
        kd, vd = 16 * rng.randint(1, 8), 16 * rng.randint(1, 8)
        if rng.random() < 0.5:
            kd = vd = 128
        n = max(1, min(n, 512 // t))
        c = _step("", n, t, ragged, shape, hv, hqk, kd, vd, rng.choice(["fp32", "fp16"]), dtype, rng.random() < 0.5)
    else:
        channels = _log(rng, 64, 8192)
        if rng.random() < 0.5:
            channels = channels // 64 * 64
        n = max(1, min(n, 2048 // t))
        c = _conv("", n, t, ragged, shape, min(channels, 2048 * 4608 // (n * t)), rng.randint(1, 8), dtype,
                  rng.random() < 0.5, rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Trees and lengths: from the case alone
# ---------------------------------------------------------------------------
def _parents(t, shape, rng):
    """Parent of each of t tokens, the root's -1; parents come first."""
    par = [-1]
    for i in range(1, t):
        if shape == "chain" or rng.random() < (0.7 if shape == "deep" else 0.25):
            par.append(i - 1)
        else:
            par.append(rng.randint(max(0, i - 12), i - 1))
    return par


def layout(case):
    """Tokens, context and parents of each request.  Ragged: odd sizes, the last of four or more requests without tokens."""
    n, t, ctx = case["n"], case["t"], case.get("ctx", 0)
    rng = random.Random("%s %d %d %d %s" % (case["op"], n, t, ctx, case["shape"]))
    ts, cs = [t] * n, [ctx] * n
    if case["ragged"]:
        ts = [t] + [rng.randint(1, t) for _ in range(n - 1)]
        cs = [ctx] + [_log(rng, 1, max(1, ctx)) - 1 for _ in range(n - 1)]
        if n >= 4:
            ts[-1] = 0
    return ts, cs, [_parents(x, case["shape"], rng) if x else [] for x in ts]


def _masks(parents):
    """Each token's ancestors and itself."""
    m = []
    for i, p in enumerate(parents):
        m.append((m[p] if p >= 0 else 0) | 1 << i)
    return m


def work(case):
    ts, cs, par = layout(case)
    total, live = sum(ts), sum(1 for t in ts if t)
    e = SIZE[case["dtype"]]
    if case["op"] == "accept":
        # a row of the target's and of the draft's probabilities for each request, two values for each token
        rows = 2 if case["drawn"] else 1
        return {"bytes": live * case["vocab"] * rows * e + total * (rows * e + 16), "flops": 4.0 * live * case["vocab"]}
    if case["op"] == "attend":
        w = case["window"] or 1 << 60
        hkv, dim = case["hkv"], case["dim"]
        keys = pairs = 0
        for t, c, p in zip(ts, cs, par):
            depth = [bin(m).count("1") - 1 for m in _masks(p)]
            keys += t + min(c, w) if t else 0
            pairs += sum(min(d + 1, w) + max(0, min(c, w - d - 1)) for d in depth)
        return {"bytes": keys * hkv * dim * 2 * 9 / 16 + 2 * total * case["hq"] * dim * e,
                "flops": 4.0 * pairs * case["hq"] * dim}
    if case["op"] == "step":
        hv, hqk, kd, vd = case["hv"], case["hqk"], case["kd"], case["vd"]
        state = hv * kd * vd * SIZE[case["pool"]]
        token = e * (2 * hqk * kd + hv * vd) + 4 * hv * (kd + 1 + vd)
        return {"bytes": (live + total) * state + total * token, "flops": 7.0 * total * hv * kd * vd}
    c, kw = case["channels"], case["width"]
    return {"bytes": (2 * total + live * (kw - 1)) * c * e + c * (kw + 1) * 4, "flops": 2.0 * kw * total * c}


# ---------------------------------------------------------------------------
# The 4-bit blocks of the cache: a value is code x scale, codes e2m1, one e4m3
# scale for 16 neighbouring channels.  Sixteen tokens of a head make a block of
# 18 * dim bytes: key codes [16][dim/2]; value codes in fragment order; key
# scales [16][dim/16]; value scales in fragment order.
# ---------------------------------------------------------------------------
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _encode(x):
    """(codes, e4m3 scale bytes) of finite x [..., dim]."""
    g = x.unflatten(-1, (-1, 16))
    s8 = (g.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
    y = g / s8.float().clamp(min=1e-9)
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    c = torch.bucketize(y.abs(), border).to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)
    return c.flatten(-2), s8.view(torch.uint8).squeeze(-1)


def _places(dim, device):
    """Byte places in a block, by token of the block: key codes, value codes [16, dim/2], key scales, value scales [16, dim/16]."""
    cb = ng = dim // 16
    key = torch.arange(16, device=device).view(16, 1)
    half, tq, j = key // 8, key % 8 // 2, key % 2
    byte = torch.arange(dim // 2, device=device).view(1, -1)
    grp = torch.arange(ng, device=device).view(1, -1)
    kc = key * (dim // 2) + byte
    vc = 8 * dim + half * (64 * cb) + (byte // cb * 4 + tq) * (2 * cb) + j * cb + byte % cb
    ks = 16 * dim + key * ng + grp
    vs = 17 * dim + (grp * 4 + tq) * 4 + half * 2 + j
    return kc, vc, ks, vs


def _fill(pages, ids, g, gain):
    """Random keys (channels times gain [heads, dim]) and values in every place of the pages `ids`."""
    heads, blocks, bytes_ = pages.shape[1:]
    dim = bytes_ // 18
    places = _places(dim, pages.device)
    for a in range(0, ids.numel(), 64):
        part = ids[a:a + 64].long()
        out = pages.new_zeros(part.numel(), heads, blocks, 18 * dim)
        shape = (part.numel(), blocks * 16, heads, dim)
        kc, ks = _encode(_randn(g, *shape) * gain)
        vc, vs = _encode(_randn(g, *shape))
        for data, place in zip((kc[..., 0::2] | (kc[..., 1::2] << 4), vc[..., 0::2] | (vc[..., 1::2] << 4), ks, vs), places):
            out[..., place] = data.unflatten(1, (blocks, 16)).permute(0, 3, 1, 2, 4)
        pages[part] = out


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


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    dt = DT[case["dtype"]]
    ts, cs, par = layout(case)
    n, total, max_t = case["n"], sum(ts), max(ts)
    cu = [0]
    for t in ts:
        cu.append(cu[-1] + t)
    # 64-bit masks as int64: bit 63 is the sign
    masks = [m - (1 << 64) if m >> 63 else m for p in par for m in _masks(p)]
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device="cuda"), "cu": _ints(cu), "max_t": max_t,
         "total": total, "tree": _ints(masks, torch.int64)}
    # for the plain forms: request and place of each token, its parent's place (padded by request), its depth
    s["req"] = _ints([r for r, t in enumerate(ts) for _ in range(t)], torch.int64)
    s["place"] = _ints([j for t in ts for j in range(t)], torch.int64)
    s["parents"] = _ints([p + [-2] * (max_t - len(p)) for p in par], torch.int64).view(n, max_t)
    s["depth"] = _ints([bin(m).count("1") - 1 for p in par for m in _masks(p)], torch.int64)
    {"accept": _prepare_accept, "attend": _prepare_attend, "step": _prepare_step, "conv": _prepare_conv}[case["op"]](
        s, case, g, dt, ts, cs, par)
    return s


def _prepare_accept(s, case, g, dt, ts, cs, par):
    n, total, vocab = case["n"], s["total"], case["vocab"]
    s["p"] = torch.empty(total, vocab, dtype=dt, device="cuda")
    s["q"] = torch.empty(total, vocab, dtype=dt, device="cuda") if case["drawn"] else None
    s["tokens"] = torch.zeros(total, dtype=torch.int32, device="cuda")
    at = 0
    for t, p in zip(ts, par):
        if not t:
            continue
        # a draft model that is close to its target: most mass on a few tokens
        logits = 3.0 * _randn(g, t, vocab)
        drafts = logits + 0.7 * _randn(g, t, vocab)
        s["p"][at:at + t] = torch.softmax(logits, -1).to(dt)
        up = _ints([max(0, x) for x in p], torch.int64)
        if case["drawn"]:
            qs = torch.softmax(drafts, -1).to(dt)
            s["q"][at:at + t] = qs
            # each token drawn from its parent's draft distribution
            noise = -torch.log(-torch.log(_rand(g, t, vocab).clamp(1e-20, 1 - 1e-7)))
            s["tokens"][at:at + t] = (torch.log(qs.float())[up] + noise).argmax(-1).int()
        else:
            # each token's children are its draft's best
            rank, seen = [], {}
            for x in p:
                rank.append(seen.get(x, 0))
                seen[x] = rank[-1] + 1
            best = drafts.topk(max(seen.values()), -1).indices
            s["tokens"][at:at + t] = best[up, _ints(rank, torch.int64)].int()
        at += t
    s["u"], s["u_last"] = _rand(g, total), _rand(g, n)
    s["accepted"], s["node"], s["token"] = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(3))
    s["path"] = torch.empty(n, s["max_t"], dtype=torch.int32, device="cuda")


def _prepare_attend(s, case, g, dt, ts, cs, par):
    n, page, dim, hkv, rot = case["n"], case["page"], case["dim"], case["hkv"], case["rot"]
    ends = [t + c for t, c in zip(ts, cs)]
    cols = -(-max(ends) // page)
    need = [-(-e // page) for e in ends]
    num = sum(need) + 3
    perm = torch.randperm(num, generator=g, device="cuda").int()
    s["table"] = torch.zeros(n, cols, dtype=torch.int32, device="cuda")
    at = 0
    for r, c in enumerate(need):
        s["table"][r, :c] = perm[at:at + c]
        at += c
    s["pages"] = torch.zeros(num, hkv, page // 16, 18 * dim, dtype=torch.uint8, device="cuda")
    # a cache as appends left it: some key channels larger than others, as in trained models
    _fill(s["pages"], perm[:at], g, torch.exp(0.5 * _randn(g, hkv, dim)))
    s["ctx"], s["max_kv"] = _ints(cs), max(ends)
    s["cos"], s["sin"] = _tables(max(ends), rot, "cuda") if rot else (None, None)
    s["q"] = (_randn(g, s["total"], case["hq"], dim) * 1.5).to(dt)
    s["o"] = torch.empty_like(s["q"])
    s["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


def _prepare_step(s, case, g, dt, ts, cs, par):
    n, total, hv, kd, vd = case["n"], s["total"], case["hv"], case["kd"], case["vd"]
    slots = n * (s["max_t"] + 1) + 1
    s["pool"] = (0.1 * _randn(g, slots, hv, kd, vd)).to(DT[case["pool"]])
    # column max_t holds the state that the step starts from, columns 0 .. max_t - 1 the tokens' snapshots
    s["slots"] = torch.randperm(slots, generator=g, device="cuda")[: n * (s["max_t"] + 1)].int().view(n, -1)
    s["accepted"] = _ints([s["max_t"] + 1] * n)
    s["q"], s["k"] = (_randn(g, total, case["hqk"], kd).to(dt) for _ in range(2))
    s["v"] = _randn(g, total, hv, vd).to(dt)
    s["a"], s["b"] = _randn(g, total, hv, kd), _randn(g, total, hv)
    s["a_log"], s["dt_bias"] = (0.5 * _randn(g, hv), 0.5 * _randn(g, hv, kd)) if case["learned"] else (None, None)
    s["o"] = torch.empty(total, hv, vd, device="cuda")


def _prepare_conv(s, case, g, dt, ts, cs, par):
    n, total, c, kw = case["n"], s["total"], case["channels"], case["width"]
    s["x"] = _randn(g, total, c).to(dt)
    s["window"] = _randn(g, n + 2, kw + 7, c).to(dt)
    s["slots"] = torch.randperm(n + 2, generator=g, device="cuda")[:n].int()
    s["accepted"] = _ints([1 + r % 8 for r in range(n)])
    s["weight"] = _randn(g, c, kw) * kw ** -0.5
    s["bias"] = 0.1 * _randn(g, c) if case["bias"] else None
    s["y"] = torch.empty_like(s["x"])


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _plain_accept(s):
    """Tokens in order, for all requests at once: a token is tested where its parent is the last one accepted.  In 64
    bits: a draw next to a border between two tokens has to fall on the same side."""
    n, t = s["parents"].shape
    vocab, dev = s["p"].shape[1], s["p"].device
    first = s["cu"][:-1].long()
    some = s["cu"][1:].long() > first
    top = max(0, s["p"].shape[0] - 1)

    def rows(x, at):
        return x[at.clamp(0, top)].double().clamp(min=0)

    req = torch.arange(n, device=dev)
    cur = torch.zeros(n, dtype=torch.int64, device=dev)
    w = rows(s["p"], first)
    z = torch.ones(n, dtype=torch.float64, device=dev)
    count = some.long()
    path = torch.full((n, t), -1, dtype=torch.int64, device=dev)
    path[:, 0] = torch.where(some, first, -1)
    for i in range(1, t):
        mine = (s["parents"][:, i] == cur) & some
        at = (first + i).clamp(0, top)
        x = s["tokens"][at].long()
        wx, u = w[req, x], s["u"][at].double()
        qc = rows(s["q"], first + cur) if s["q"] is not None else None
        yes = mine & (u * (qc[req, x] if qc is not None else 1.0) * z < wx)
        no = mine & ~yes
        # rejected: what the target has more than the draft, or without a draft distribution the others
        if qc is not None:
            left = (w - z.unsqueeze(1) * qc).clamp(min=0)
            zl = left.sum(-1)
        else:
            left = w.clone()
            left[req, x] = 0
            zl = z - wx
        w = torch.where(yes.unsqueeze(1), rows(s["p"], at), torch.where(no.unsqueeze(1), left, w))
        z = torch.where(yes, 1.0, torch.where(no, zl, z))
        cur = torch.where(yes, i, cur)
        path[req, count.clamp(max=t - 1)] = torch.where(yes, at, path[req, count.clamp(max=t - 1)])
        count = count + yes
    # nothing left: from the target's own
    w = torch.where((w.sum(-1) > 0).unsqueeze(1), w, rows(s["p"], first + cur))
    cum = w.cumsum(-1)
    over = (cum > s["u_last"].double().unsqueeze(1) * cum[:, -1:]) & (w > 0)
    ids = torch.arange(vocab, device=dev)
    token = torch.where(over, ids, vocab).amin(-1)
    token = torch.where(token < vocab, token, torch.where(w > 0, ids, -1).amax(-1))
    return {"accepted": count.int(), "node": torch.where(some, cur + 1, 0).int(), "path": path.int(),
            "token": torch.where(some, token, -1).int()}


def _plain_attend(s):
    c = s["case"]
    n, hq, hkv, dim, page, t = c["n"], c["hq"], c["hkv"], c["dim"], c["page"], s["max_t"]
    grp, dev = hq // hkv, s["q"].device
    req, place = s["req"], s["place"]
    pos = s["ctx"].long()[req] + s["depth"]
    cos, sin = (s["cos"][pos], s["sin"][pos]) if c["rot"] else (None, None)
    q = _rotate(s["q"].float(), cos, sin, c["rot"], c["inter"])
    qp = q.new_zeros(n, t, hq, dim)
    qp[req, place] = q
    qp = qp.view(n, t, hkv, grp, dim).permute(0, 2, 1, 3, 4).reshape(n, hkv, t * grp, dim)
    cols = -(-s["max_kv"] // page)
    blocks = s["pages"][s["table"][:, :cols].long()].transpose(1, 2).reshape(n, hkv, -1, 18 * dim)
    kc, vc, ks, vs = _places(dim, dev)
    lut = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float32, device=dev)
    byte = torch.arange(256, device=dev)
    pair = torch.stack((lut[byte & 15], lut[byte >> 4]), -1)

    def rows(codes, scales):
        v = pair[blocks[..., codes].int()].flatten(-2).unflatten(-1, (-1, 16))
        v = v * blocks[..., scales].view(torch.float8_e4m3fn).float().unsqueeze(-1)
        return v.flatten(-2).flatten(2, 3)

    # what a token sees: the context, and the tokens of its mask; of both the last `window` positions
    keys = torch.arange(blocks.shape[2] * 16, device=dev)
    ctx = s["ctx"].long().view(n, 1, 1)
    before = (keys < ctx).expand(n, t, -1)
    dp = torch.zeros(n, t, dtype=torch.int64, device=dev)
    dp[req, place] = s["depth"]
    bits = torch.zeros(n, t, dtype=torch.int64, device=dev)
    bits[req, place] = s["tree"]
    own_place = keys - ctx
    inside = (own_place >= 0) & (own_place < t)
    node = own_place.clamp(0, t - 1)
    mine = inside & ((bits.unsqueeze(-1) >> node) & 1).bool()
    if c["window"]:
        before = before & (keys > ctx + dp.unsqueeze(-1) - c["window"])
        mine = mine & (dp.gather(1, node.squeeze(1)).unsqueeze(1) > dp.unsqueeze(-1) - c["window"])
    seen = (before | mine).unsqueeze(2).expand(n, t, grp, -1).reshape(n, 1, t * grp, -1)
    score = torch.matmul(qp, rows(kc, ks).transpose(-1, -2)) * dim ** -0.5
    score = score.masked_fill(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    o = torch.matmul(p, rows(vc, vs)) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(n, hkv, t, grp, dim).permute(0, 2, 1, 3, 4).reshape(n, t, hq, dim)
    return {"o": o[req, place].to(s["o"].dtype)}


def _plain_step(s):
    c = s["case"]
    n, t, hv, kd, vd = c["n"], s["max_t"], c["hv"], c["kd"], c["vd"]
    rep = hv // c["hqk"]

    def unit(x):
        x = x.float()
        return (x * torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6)).repeat_interleave(rep, 1)

    a = s["a"] if s["dt_bias"] is None else s["a"] + s["dt_bias"]
    soft = torch.nn.functional.softplus(a)
    alpha = torch.exp(-soft if s["a_log"] is None else -torch.exp(s["a_log"]).view(hv, 1) * soft)
    q, k, v, beta = unit(s["q"]), unit(s["k"]), s["v"].float(), torch.sigmoid(s["b"])
    req, place = s["req"], s["place"]

    def padded(x):
        y = x.new_zeros(n, t, *x.shape[1:])
        y[req, place] = x
        return y

    q, k, v, alpha, beta = (padded(x) for x in (q, k, v, alpha, beta))
    states = torch.empty(n, t + 1, hv, kd, vd, device=q.device)
    states[:, t] = s["pool"][s["slots"][:, t].long()].float()
    o = torch.empty(n, t, hv, vd, device=q.device)
    ids = torch.arange(n, device=q.device)
    up = torch.where(s["parents"] >= 0, s["parents"], t)
    for j in range(t):
        S = states[ids, up[:, j]] * alpha[:, j].unsqueeze(-1)
        kj = k[:, j].unsqueeze(-1)
        u = (S * kj).sum(-2)
        S = S + kj * (beta[:, j].unsqueeze(-1) * (v[:, j] - u)).unsqueeze(-2)
        states[:, j] = S
        o[:, j] = (S * q[:, j].unsqueeze(-1)).sum(-2) * kd ** -0.5
    s["pool"][s["slots"][req, place].long()] = states[req, place].to(s["pool"].dtype)
    return {"o": o[req, place], "pool": s["pool"]}


def _plain_conv(s):
    c = s["case"]
    kw, t, n = c["width"], s["max_t"], c["n"]
    req, place = s["req"], s["place"]
    # rows of inputs behind the history, by request: history entry i at i, token j at kw - 1 + j
    hist = torch.arange(kw - 1, device=req.device) + (s["accepted"].long() - 1).unsqueeze(1)
    z = torch.zeros(n, kw - 1 + t, c["channels"], device=req.device)
    z[:, : kw - 1] = s["window"][s["slots"].long().unsqueeze(1), hist].float()
    z[req, kw - 1 + place] = s["x"].float()
    up = s["parents"][req]  # [total, t]
    at = place.clone()      # the tap's place: a token, or -1 - i for the i-th entry of the history from its end
    y = torch.zeros_like(s["x"], dtype=torch.float32)
    for i in range(kw - 1, -1, -1):
        y = y + s["weight"][:, i] * z[req, kw - 1 + at]
        above = up.gather(1, at.clamp(min=0).unsqueeze(1)).squeeze(1)
        at = torch.where(at >= 0, above, (at - 1).clamp(min=1 - kw))
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["silu"]:
        y = y * torch.sigmoid(y)
    return {"y": y.to(s["x"].dtype)}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"accept": _plain_accept, "attend": _plain_attend, "step": _plain_step, "conv": _plain_conv}[c["op"]](s)
    if c["op"] == "accept":
        lib().kda_accept(s["p"], s["tokens"], s["u"], s["u_last"], s["accepted"], s["node"], s["path"], s["token"],
                         s["status"], q=s["q"], tree=s["tree"], cu_seqlens=s["cu"], max_t=s["max_t"])
        return {k: s[k] for k in ("accepted", "node", "path", "token")}
    if c["op"] == "attend":
        lib().kda_kv4_attend_tree(s["pages"], s["table"], s["ctx"], s["q"], s["tree"], s["o"], s["workspace"],
                                  s["status"], cu_seqlens=s["cu"], max_t=s["max_t"], cos=s["cos"], sin=s["sin"],
                                  interleaved=c["inter"], window=c["window"])
        return {"o": s["o"]}
    if c["op"] == "step":
        lib(s["pool"].dtype).kda_step_tree(s["pool"], s["slots"], s["q"], s["k"], s["v"], s["a"], s["b"], s["tree"],
                                           s["o"], s["status"], cu_seqlens=s["cu"], max_t=s["max_t"],
                                           accepted=s["accepted"], a_log=s["a_log"], dt_bias=s["dt_bias"])
        return {"o": s["o"], "pool": s["pool"]}
    lib().kda_conv_step_tree(s["window"], s["slots"], s["x"], s["weight"], s["tree"], s["y"], s["status"],
                             bias=s["bias"], cu_seqlens=s["cu"], max_t=s["max_t"], accepted=s["accepted"],
                             silu=c["silu"])
    return {"y": s["y"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, request by request
# ---------------------------------------------------------------------------
def _exact_accept(s, ts, par):
    n = len(ts)
    out = {"accepted": torch.zeros(n, dtype=torch.int32), "node": torch.zeros(n, dtype=torch.int32),
           "path": torch.full((n, s["max_t"]), -1, dtype=torch.int32), "token": torch.full((n,), -1, dtype=torch.int32)}
    at = 0
    for r, (t, p) in enumerate(zip(ts, par)):
        if not t:
            continue
        node, path, i = 0, [at], 1
        weight, mass = s["p"][at].double(), 1.0
        while i < t:
            if p[i] != node:
                i += 1
                continue
            x, u = int(s["tokens"][at + i]), float(s["u"][at + i])
            held = float(weight[x])
            q = s["q"][at + node].double() if s["q"] is not None else None
            if u * (float(q[x]) if q is not None else 1.0) * mass < held:
                node = i
                path.append(at + i)
                weight, mass = s["p"][at + i].double(), 1.0
            elif q is None:
                weight = weight.clone()
                weight[x] = 0.0
                mass -= held
            else:
                weight = torch.relu(weight - mass * q)
                mass = float(weight.sum())
            i += 1
        if not float(weight.sum()) > 0:
            weight = s["p"][at + node].double()
        kept = torch.nonzero(weight).flatten()
        cum = torch.cumsum(weight[kept], 0)
        k = int(torch.searchsorted(cum, s["u_last"][r].double() * cum[-1], right=True))
        out["accepted"][r], out["node"][r] = len(path), node + 1
        out["path"][r, : len(path)] = torch.tensor(path, dtype=torch.int32)
        out["token"][r] = int(kept[min(k, kept.numel() - 1)])
        at += t
    return {k: v.cuda() for k, v in out.items()}


def _exact_attend(s, case, ts, cs, par):
    hkv, dim, page, rot = case["hkv"], case["dim"], case["page"], case["rot"]
    grp, w = case["hq"] // hkv, case["window"] or 1 << 60
    q = s["q"].double()
    if rot:
        pos = (s["ctx"].long()[s["req"]] + s["depth"]).double()
        i = torch.arange(rot // 2, device="cuda")
        ang = pos.view(-1, 1) * (10000.0 ** (-2.0 * i.double() / rot)).view(1, -1)
        # the tables are inputs in 32 bits
        co, si = ang.cos().float().double().unsqueeze(1), ang.sin().float().double().unsqueeze(1)
        a, b = (2 * i, 2 * i + 1) if case["inter"] else (i, i + rot // 2)
        x = q.clone()
        x[..., a], x[..., b] = q[..., a] * co - q[..., b] * si, q[..., b] * co + q[..., a] * si
        q = x
    grid = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
    o, at = torch.zeros_like(q), 0
    for r, (t, ctx, p) in enumerate(zip(ts, cs, par)):
        if not t:
            continue
        end = ctx + t
        depth = []
        for j in range(t):
            depth.append(depth[p[j]] + 1 if p[j] >= 0 else 0)
        see = torch.zeros(t, end, dtype=torch.bool)
        for j in range(t):
            see[j, max(0, ctx + depth[j] - w + 1):ctx] = True
            i = j
            while i >= 0:
                see[j, ctx + i] = depth[i] > depth[j] - w
                i = p[i]
        hide = ~see.cuda().unsqueeze(1)
        for h in range(hkv):
            b = s["pages"][s["table"][r, : -(-end // page)].long(), h].reshape(-1, 18 * dim)
            codes_k = b[:, : 8 * dim].reshape(-1, 16, dim // 2)
            # value codes: [half][channel eighth][quad][token of a pair][bytes] of each block
            codes_v = b[:, 8 * dim: 16 * dim].reshape(-1, 2, 8, 4, 2, dim // 16).permute(0, 1, 3, 4, 2, 5)
            codes_v = codes_v.reshape(-1, 16, dim // 2)
            sk = b[:, 16 * dim: 17 * dim].reshape(-1, 16, dim // 16)
            sv = b[:, 17 * dim:].reshape(-1, dim // 16, 4, 2, 2).permute(0, 3, 2, 4, 1).reshape(-1, 16, dim // 16)

            def rows(codes, scales):
                c = torch.stack((codes & 15, codes >> 4), -1).reshape(-1, dim)[:end].long()
                f = scales.contiguous().view(torch.float8_e4m3fn).double().reshape(-1, dim // 16)[:end]
                return torch.where(c >= 8, -grid[c & 7], grid[c & 7]) * f.repeat_interleave(16, -1)

            x = q[at:at + t, h * grp:(h + 1) * grp]
            score = torch.einsum("tgd,pd->tgp", x, rows(codes_k, sk)) / dim ** 0.5
            o[at:at + t, h * grp:(h + 1) * grp] = torch.einsum(
                "tgp,pd->tgd", torch.softmax(score.masked_fill(hide, float("-inf")), -1), rows(codes_v, sv))
        at += t
    return {"o": o}


def _exact_step(s, case, ts, par):
    hv, kd = case["hv"], case["kd"]
    head = torch.arange(hv, device="cuda") // (hv // case["hqk"])
    pool, o, at = s["pool"].double(), torch.zeros_like(s["o"], dtype=torch.float64), 0
    out = pool.clone()
    for r, (t, p) in enumerate(zip(ts, par)):
        states = []
        for j in range(t):
            k, q = s["k"][at + j].double()[head], s["q"][at + j].double()[head]
            k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
            q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6)
            a = s["a"][at + j].double()
            if case["learned"]:
                decay = (1 + torch.exp(a + s["dt_bias"].double())) ** -torch.exp(s["a_log"].double()).unsqueeze(1)
            else:
                decay = 1 / (1 + torch.exp(a))
            S = (states[p[j]] if p[j] >= 0 else pool[s["slots"][r, s["max_t"]].long()]) * decay.unsqueeze(-1)
            u = torch.einsum("hkv,hk->hv", S, k)
            rate = (1 / (1 + torch.exp(-s["b"][at + j].double()))).unsqueeze(-1)
            S = S + torch.einsum("hk,hv->hkv", k, rate * (s["v"][at + j].double() - u))
            states.append(S)
            out[s["slots"][r, j].long()] = S
            o[at + j] = torch.einsum("hkv,hk->hv", S, q) / kd ** 0.5
        at += t
    return {"o": o, "pool": out}


def _exact_conv(s, case, ts, par):
    kw, at = case["width"], 0
    y = torch.zeros_like(s["x"], dtype=torch.float64)
    for r, (t, p) in enumerate(zip(ts, par)):
        first = int(s["accepted"][r]) - 1
        past = list(s["window"][int(s["slots"][r]), first:first + kw - 1].double())
        lines = []
        for j in range(t):
            lines.append((lines[p[j]] if p[j] >= 0 else past) + [s["x"][at + j].double()])
            taps = lines[j][len(lines[j]) - kw:]
            v = sum(s["weight"][:, i].double() * taps[i] for i in range(kw))
            if s["bias"] is not None:
                v = v + s["bias"].double()
            y[at + j] = v / (1 + torch.exp(-v)) if case["silu"] else v
        at += t
    return {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    ts, cs, par = layout(case)
    if case["op"] == "accept":
        return _exact_accept(s, ts, par)
    if case["op"] == "attend":
        return _exact_attend(s, case, ts, cs, par)
    if case["op"] == "step":
        return _exact_step(s, case, ts, par)
    return _exact_conv(s, case, ts, par)
