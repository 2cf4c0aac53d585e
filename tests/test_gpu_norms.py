"""kda_head_norm and kda_block_norm against fp64."""
import pytest
import torch

import kda_linear_attention_gated_gb300 as kda
from kda_linear_attention_gated_gb300 import BlockNormArgs, HeadNormArgs

import _layer_ref as ref

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
P = 0x7F0000100000
# fp32 work behind one rounding of the result: the mean (a sum of n terms in a
# tree of depth about 8 + n / threads), 1 / sqrt, the exponential and the
# reciprocal of a sigmoid, and the products: 24 half steps cover them all
WORK = 24 * 2.0 ** -24


@pytest.fixture(scope="module")
def lib(built_libs):
    return kda.KdaLibrary(torch.float32)


def test_head_norm_refusals(lib):
    import ctypes

    def call(flags=0, **kw):
        d = dict(total=4, heads=2, dim=128, o_dtype=kda.KDA_F32, dtype=kda.KDA_BF16, activation=1, eps=1e-6, reserved=0, gate_stride=256,
                 o=P, gate=P, weight=P, y=P)
        d.update(kw)
        return lib.lib.kda_head_norm(ctypes.byref(HeadNormArgs(*d.values())), flags, None)

    for kw, code in [(dict(total=-1), kda.KDA_ERR_ARG), (dict(heads=0), kda.KDA_ERR_SHAPE), (dict(dim=0), kda.KDA_ERR_SHAPE),
                     (dict(dim=12), kda.KDA_ERR_SHAPE), (dict(dim=264), kda.KDA_ERR_SHAPE), (dict(o_dtype=4), kda.KDA_ERR_DTYPE_UNSUPPORTED),
                     (dict(dtype=-1), kda.KDA_ERR_DTYPE_UNSUPPORTED), (dict(activation=3), kda.KDA_ERR_ARG), (dict(eps=-1.0), kda.KDA_ERR_ARG),
                     (dict(eps=float("nan")), kda.KDA_ERR_ARG), (dict(reserved=2), kda.KDA_ERR_ARG), (dict(gate_stride=255), kda.KDA_ERR_SHAPE),
                     (dict(gate_stride=260), kda.KDA_ERR_ALIGN), (dict(o=None), kda.KDA_ERR_NULL), (dict(weight=None), kda.KDA_ERR_NULL),
                     (dict(y=P + 8), kda.KDA_ERR_ALIGN), (dict(gate=P + 2), kda.KDA_ERR_ALIGN), (dict(flags=2), kda.KDA_ERR_ARG),
                     (dict(total=0), kda.KDA_OK)]:
        assert call(**kw) == code, kw
    assert lib.lib.kda_head_norm(None, 0, None) == kda.KDA_ERR_NULL


def test_block_norm_refusals(lib):
    import ctypes

    def call(flags=0, **kw):
        d = dict(total=4, hidden=64, dtype=kda.KDA_BF16, residual_dtype=kda.KDA_F32, activation=1, eps=1e-6, residual_scale=1.0, branch_scale=1.0,
                 y_stride=64, gate_stride=64, residual=P, y=P, gate=P, w_post=P, scale=P, w_pre=P, residual_out=P, x=P)
        d.update(kw)
        return lib.lib.kda_block_norm(ctypes.byref(BlockNormArgs(*d.values())), flags, None)

    for kw, code in [(dict(total=-1), kda.KDA_ERR_ARG), (dict(hidden=0), kda.KDA_ERR_SHAPE), (dict(hidden=kda.KDA_BLOCK_NORM_MAX + 1), kda.KDA_ERR_SHAPE),
                     (dict(dtype=3), kda.KDA_ERR_DTYPE_UNSUPPORTED), (dict(residual_dtype=kda.KDA_F16), kda.KDA_ERR_DTYPE_UNSUPPORTED),
                     (dict(activation=-1), kda.KDA_ERR_ARG), (dict(eps=-1.0), kda.KDA_ERR_ARG), (dict(y_stride=63), kda.KDA_ERR_SHAPE),
                     (dict(gate_stride=1), kda.KDA_ERR_SHAPE), (dict(residual=None), kda.KDA_ERR_NULL), (dict(residual_out=None), kda.KDA_ERR_NULL),
                     (dict(y=None), kda.KDA_ERR_NULL), (dict(y=None, gate=None, w_post=None, scale=None, x=None), kda.KDA_ERR_NULL),
                     (dict(y=P + 1), kda.KDA_ERR_ALIGN), (dict(residual=P + 2), kda.KDA_ERR_ALIGN), (dict(w_pre=P + 2), kda.KDA_ERR_ALIGN),
                     (dict(flags=4), kda.KDA_ERR_ARG), (dict(total=0), kda.KDA_OK)]:
        assert call(**kw) == code, kw
    assert lib.lib.kda_block_norm(None, 0, None) == kda.KDA_ERR_NULL


def close(got, want, dtype, mag=None, what=""):
    """One rounding to dtype on top of the fp32 work; subnormals of a 16-bit type by their own step."""
    got = got.cpu().double()
    step = ref.half_step(dtype)
    lim = step * want.abs() + WORK * (want.abs() if mag is None else mag) * (1 + step)
    if dtype == F16:
        lim = torch.clamp(lim, min=2.0 ** -25 * (1 + 2.0 ** -10))
    assert torch.equal(got.isnan(), want.isnan()), what
    bad = (got - want).abs() > lim
    assert not bad.any(), f"{what}: worst {((got - want).abs() / lim).nan_to_num(0).max():.3g} of the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("total,heads,dim,src,dtype,kind,strided", [
    (1, 1, 8, F32, F32, 1, False), (64, 12, 128, F32, BF16, 1, False), (7, 3, 80, F32, F16, 2, True), (5, 1, 256, BF16, BF16, 0, False),
    (33, 5, 48, F16, F32, 1, True), (301, 4, 16, BF16, F16, None, False), (3, 2, 136, F16, BF16, 2, False), (1, 12, 128, BF16, F32, None, False),
])
def test_head_norm_against_fp64(lib, total, heads, dim, src, dtype, kind, strided):
    g = torch.Generator().manual_seed(dim)
    o = (torch.randn(total, heads, dim, generator=g) * 0.1).to(src)
    o[0, 0] = 0.0
    w = 1 + 0.2 * torch.randn(dim, generator=g)
    wide = (torch.randn(total, heads + 1, dim, generator=g) * 3).to(dtype)
    gate = None if kind is None else wide[:, 1:] if strided else wide[:, 1:].contiguous()
    y = torch.full((total, heads, dim), float("nan"), dtype=dtype, device="cuda")
    gg = None if kind is None else wide.cuda()[:, 1:] if strided else gate.cuda()
    lib.kda_head_norm(o.cuda(), w.cuda(), y, gate=gg, activation=kind or 0, eps=1e-5)
    close(y, ref.head_norm(o, w, gate, kind or 0, 1e-5), dtype)


@pytest.mark.gpu
def test_head_norm_in_place_and_not_finite(lib):
    o = torch.randn(6, 2, 64)
    o[1, 0, 3], o[2, 1, 5] = float("nan"), float("inf")
    gate = torch.randn(6, 2, 64)
    gate[4, 0, 0], gate[4, 0, 1] = 200.0, -200.0
    w = torch.ones(64)
    y = o.cuda()
    lib.kda_head_norm(y, w.cuda(), y, gate=gate.cuda())
    got = y.cpu()
    assert got[1, 0].isnan().all() and got[2, 1].isnan().sum() == 1 and got[[0, 3, 4, 5]].isfinite().all()
    want = ref.head_norm(o, w, gate, 1, 1e-6)
    close(got[[0, 3, 4, 5]], want[[0, 3, 4, 5]], F32, mag=want[[0, 3, 4, 5]].abs() + 2.0 ** -100)


def run_block(lib, total, hidden, dtype, res, kind=1, post=True, scale=True, pre=True, out=True, strided=False, offset=0, in_place=False, seed=0,
              edit=None):
    g = torch.Generator().manual_seed(seed + hidden)
    mk = lambda *s: torch.randn(*s, generator=g)  # noqa: E731

    def dev(t):   # at an element offset of its buffer: rows that do not start on 16 bytes
        buf = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
        v = buf[offset:].view(t.shape)
        v.copy_(t)
        return v

    wide = (mk(total, 2 * hidden + 8) * 0.5).to(dtype)
    gate_all = (mk(total, 2 * hidden + 8) * 2).to(dtype)
    residual = (mk(total, hidden) * 2).to(res)
    if edit is not None:
        edit(wide, residual)
    y, gate = wide[:, 8:8 + hidden], gate_all[:, :hidden]
    wp = 1 + 0.2 * mk(hidden) if post else None
    sc = 0.5 + 0.2 * mk(hidden) if scale else None
    wq = 1 + 0.2 * mk(hidden) if pre else None
    yd = wide.cuda()[:, 8:8 + hidden] if strided else dev(y.contiguous())
    gd = None if kind is None else gate_all.cuda()[:, :hidden] if strided else dev(gate.contiguous())
    rd = dev(residual)
    ro = rd if in_place else dev(torch.full_like(residual, float("nan")))
    x = dev(torch.full((total, hidden), float("nan"), dtype=dtype)) if out else None
    cu = lambda t: None if t is None else dev(t)  # noqa: E731
    lib.kda_block_norm(rd, yd, ro, w_post=cu(wp), gate=gd, activation=kind or 0, scale=cu(sc), w_pre=cu(wq), x=x, residual_scale=0.9,
                       branch_scale=-0.7, eps=1e-5)
    f = lambda v: torch.tensor(v, dtype=F32).double().item()  # noqa: E731
    h, mag, xr = ref.block_norm(residual, y, wp, None if kind is None else gate, kind or 0, sc, wq, f(0.9), f(-0.7), f(1e-5))
    close(ro, h, res, mag, "residual")
    if out:
        # the norm carries h's error: relative to |w| mag / rms(h)
        w = torch.ones(hidden).double() if wq is None else wq.double().abs()
        inv = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-5)
        close(x, xr, dtype, xr.abs() + w * mag * inv + (w * h.abs() * inv) * ((mag * h.abs()).mean(-1, keepdim=True) * inv * inv), "x")


@pytest.mark.gpu
@pytest.mark.parametrize("total,hidden,dtype,res", [
    (1, 1, F32, F32), (3, 7, BF16, BF16), (64, 4096, BF16, BF16), (5, 4096, BF16, F32), (2, 8200, F16, F16), (2, 16384, F16, F32),
    (9, 2049, F32, F32), (2, 12001, BF16, F32), (3, 16384, F32, F32), (700, 64, F16, F16), (4, 1000, BF16, BF16), (1000, 1536, BF16, F32),
])
def test_block_norm_against_fp64(lib, total, hidden, dtype, res):
    run_block(lib, total, hidden, dtype, res)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(kind=None), dict(kind=0), dict(kind=2), dict(post=False), dict(scale=False), dict(pre=False), dict(out=False),
                                dict(post=False, kind=None, scale=False), dict(strided=True), dict(in_place=True), dict(offset=1), dict(offset=3, strided=True),
                                dict(post=False, out=False)])
@pytest.mark.parametrize("dtype,res", [(BF16, F32), (F16, F16)])
def test_block_norm_options(lib, kw, dtype, res):
    run_block(lib, 321, 320, dtype, res, **kw)
    run_block(lib, 3, 4096, dtype, res, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("total,hidden,dtype,res,kw", [
    (1700, 9, BF16, BF16, {}), (1300, 77, F16, F32, {}), (2500, 130, F32, F32, dict(in_place=True)), (700, 1001, BF16, F32, dict(in_place=True)),
    (320, 4101, F16, F16, dict(kind=2)), (310, 8191, F32, F32, dict(kind=None)), (5, 3, BF16, F32, {}), (8, 8190, BF16, BF16, dict(post=False, out=False)),
    (33, 101, BF16, BF16, dict(strided=True)), (9, 5, F32, F32, dict(strided=True, out=False)), (2000, 15, F16, F32, dict(kind=0, scale=False, pre=False)),
])
def test_block_norm_of_widths_that_are_no_multiple_of_eight(lib, total, hidden, dtype, res, kw):
    """Rows that begin anywhere in a 16-byte vector, several to a CTA: neighbours' channels are neither summed nor written."""
    run_block(lib, total, hidden, dtype, res, **kw)


@pytest.mark.gpu
def test_block_norm_odd_width_keeps_not_finite_rows_apart(lib):
    y, r = torch.randn(40, 37), torch.randn(40, 37)
    y[7, 36], y[9, 0], r[20, 5] = float("nan"), float("inf"), float("nan")
    ro, x = torch.empty(40, 37, device="cuda"), torch.empty(40, 37, device="cuda")
    w = torch.ones(37, device="cuda")
    lib.kda_block_norm(r.cuda(), y.cuda(), ro, w_post=w, w_pre=w, x=x)
    bad = sorted(set((~x.cpu().isfinite()).any(1).nonzero().flatten().tolist()))
    assert bad == [7, 9, 20]


@pytest.mark.gpu
def test_block_norm_of_the_residual_alone(lib):
    r = torch.randn(5, 264)
    x = torch.empty(5, 264, dtype=BF16, device="cuda")
    w = torch.rand(264) + 0.5
    lib.kda_block_norm(r.cuda(), None, None, w_pre=w.cuda(), x=x)
    h, mag, xr = ref.block_norm(r, None, None, None, 0, None, w, 1, 1, 1e-6)
    close(x, xr, BF16)


@pytest.mark.gpu
def test_block_norm_zero_rows_and_not_finite_rows(lib):
    """A zero row stays zero; a NaN or an infinity stays in its own row."""
    def edit(y, residual):
        y[0], residual[0] = 0.0, 0.0
    run_block(lib, 4, 512, BF16, F32, edit=edit)
    y, r = torch.randn(4, 512), torch.randn(4, 512)
    y[1, 5], r[2, 7] = float("nan"), float("inf")
    ro, x = torch.empty(4, 512, device="cuda"), torch.empty(4, 512, device="cuda")
    w = torch.ones(512, device="cuda")
    lib.kda_block_norm(r.cuda(), y.cuda(), ro, w_post=w, w_pre=w, x=x)
    assert ro[1].isnan().all() and x[1].isnan().all() and x[2].isnan().sum() == 1
    assert ro[[0, 3]].isfinite().all() and x[[0, 3]].isfinite().all()


@pytest.mark.gpu
def test_norms_in_a_graph_with_programmatic_launch(lib):
    """recurrence output -> head norm -> block norm captured on a side stream."""
    g = torch.Generator().manual_seed(2)
    o, gate = torch.randn(9, 4, 64, generator=g).cuda(), torch.randn(9, 4, 64, generator=g).to(BF16).cuda()
    w1, w2 = torch.rand(64, generator=g).cuda(), torch.rand(256, generator=g).cuda()
    res = torch.randn(9, 256, generator=g).to(BF16).cuda()
    outs = []
    for flags in (0, kda.KDA_LAUNCH_PDL):
        y, ro, x = torch.empty(9, 4, 64, dtype=BF16, device="cuda"), torch.empty_like(res), torch.empty_like(res)

        def step(stream=None):
            lib.kda_head_norm(o, w1, y, gate=gate, stream=stream, flags=flags)
            lib.kda_block_norm(res, y.view(9, 256), ro, w_post=w2, w_pre=w2, x=x, stream=stream, flags=flags)

        if flags:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step(side)
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        outs.append((y, ro, x))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
