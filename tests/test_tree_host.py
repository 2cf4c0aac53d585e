"""A speculative step over a tree of drafted tokens, on the host: refusals before any launch, the binding's structs
and checks, and the references against other definitions (no GPU)."""
import ctypes

import pytest
import torch

import kda_linear_attention_gated_gb300 as kda
from kda_linear_attention_gated_gb300 import AcceptArgs, ConvArgs, ConvWindowDesc, PoolDesc, StepArgs

import _tree_ref as ref
from test_gpu_kv4 import append_args, attend_args, cache_desc

P = 0x7F0000100000
PAIRS = [(kda._PACK_POOL, kda.PoolDesc), (kda._PACK_STEP, kda.StepArgs), (kda._PACK_CONV_WINDOW, kda.ConvWindowDesc),
         (kda._PACK_CONV, kda.ConvArgs), (kda._PACK_ACCEPT, kda.AcceptArgs)]


@pytest.fixture(scope="module")
def lib(built_libs):
    return kda.KdaLibrary(torch.float32)


@pytest.mark.parametrize("packer,mirror", PAIRS, ids=[m.__name__ for _, m in PAIRS])
def test_packed_arguments_have_the_structs_layout(packer, mirror):
    assert packer.size == ctypes.sizeof(mirror)
    values = list(range(1, 1 + len(mirror._fields_)))
    got = mirror.from_buffer_copy(packer.pack(*values))
    assert [getattr(got, name) for name, _ in mirror._fields_] == values


def make(kind, fields, /, **kw):
    fields = dict(fields)
    fields.update(kw)
    return kind(*fields.values())


POOL = dict(base=P, dtype=kda.KDA_F32, hv=4, k=64, v=64, num_slots=8, slot_stride=4 * 64 * 64)
STEP = dict(n=2, total=6, max_t=3, h_qk=2, num_cols=4, in_place=0, qkv_dtype=kda.KDA_BF16, reserved=0, cu_seqlens=None, slot_table=P,
            accepted=None, reset=None, q=P, k=P, v=P, a=P, b=P, a_log=None, dt_bias=None, o=P)
WIN = dict(base=P, dtype=kda.KDA_BF16, channels=96, state_len=5, reserved=0, num_slots=4, slot_stride=480)
CONV = dict(n=2, total=6, max_t=3, kernel_width=4, activation=1, reserved=0, cu_seqlens=None, conv_slot=P, accepted=None, reset=None,
            x=P, weight=P, bias=None, y=P)
ACCEPT = dict(n=2, total=6, max_t=3, vocab=100, dtype=kda.KDA_F32, reserved=0, p_stride=100, q_stride=100, cu_seqlens=None, tree=P, p=P,
              q=P, tokens=P, u=P, u_last=P, accepted=P, node=P, path=P, token=P)
E = kda


def test_step_tree_refusals(lib):
    call = lib.kda_step_tree_raw
    for kw, code in ((dict(base=None), E.KDA_ERR_NULL), (dict(dtype=kda.KDA_F16), E.KDA_ERR_DTYPE_MISMATCH),
                     (dict(dtype=kda.KDA_BF16), E.KDA_ERR_DTYPE_UNSUPPORTED), (dict(k=72), E.KDA_ERR_SHAPE), (dict(v=0), E.KDA_ERR_SHAPE),
                     (dict(base=P + 4), E.KDA_ERR_ALIGN), (dict(slot_stride=4 * 64 * 64 - 4), E.KDA_ERR_SHAPE)):
        assert call(make(PoolDesc, POOL, **kw), make(StepArgs, STEP), P, P, None) == code, kw
    for kw, code in ((dict(n=-1), E.KDA_ERR_ARG), (dict(reserved=1), E.KDA_ERR_ARG), (dict(in_place=1), E.KDA_ERR_ARG),
                     (dict(total=5), E.KDA_ERR_SHAPE), (dict(h_qk=3), E.KDA_ERR_SHAPE), (dict(h_qk=0), E.KDA_ERR_SHAPE),
                     (dict(num_cols=2), E.KDA_ERR_SHAPE), (dict(max_t=65, total=130, num_cols=70), E.KDA_ERR_SHAPE),
                     (dict(qkv_dtype=7), E.KDA_ERR_DTYPE_UNSUPPORTED), (dict(q=None), E.KDA_ERR_NULL), (dict(o=None), E.KDA_ERR_NULL),
                     (dict(slot_table=None), E.KDA_ERR_NULL), (dict(a=P + 8), E.KDA_ERR_ALIGN), (dict(k=P + 8), E.KDA_ERR_ALIGN),
                     (dict(accepted=P + 1), E.KDA_ERR_ALIGN), (dict(dt_bias=P + 2), E.KDA_ERR_ALIGN)):
        assert call(make(PoolDesc, POOL), make(StepArgs, STEP, **kw), P, P, None) == code, kw
    assert call(make(PoolDesc, POOL), make(StepArgs, STEP), None, P, None) == E.KDA_ERR_NULL
    assert call(make(PoolDesc, POOL), make(StepArgs, STEP), P + 4, P, None) == E.KDA_ERR_ALIGN
    assert call(make(PoolDesc, POOL), make(StepArgs, STEP), P, None, None) == E.KDA_ERR_NULL
    for flags in (kda.KDA_LAUNCH_PDL_EARLY_STATE, kda.KDA_LAUNCH_TEST_WITHHOLD_STATE):
        assert call(make(PoolDesc, POOL), make(StepArgs, STEP), P, P, None, flags) == E.KDA_ERR_ARG
    assert call(make(PoolDesc, POOL), make(StepArgs, STEP, n=0, total=0), None, None, None) == E.KDA_OK
    assert lib.lib.kda_step_tree(ctypes.byref(make(PoolDesc, POOL)), None, P, P, 0, None) == E.KDA_ERR_NULL


def test_conv_step_tree_refusals(lib):
    call = lib.kda_conv_step_tree_raw
    for kw, code in ((dict(base=None), E.KDA_ERR_NULL), (dict(dtype=5), E.KDA_ERR_DTYPE_UNSUPPORTED), (dict(reserved=1), E.KDA_ERR_ARG),
                     (dict(channels=0), E.KDA_ERR_SHAPE), (dict(state_len=2), E.KDA_ERR_SHAPE), (dict(state_len=33), E.KDA_ERR_SHAPE),
                     (dict(slot_stride=479), E.KDA_ERR_SHAPE), (dict(base=P + 1), E.KDA_ERR_ALIGN)):
        assert call(make(ConvWindowDesc, WIN, **kw), make(ConvArgs, CONV), P, P, None) == code, kw
    for kw, code in ((dict(total=-1), E.KDA_ERR_ARG), (dict(activation=2), E.KDA_ERR_ARG), (dict(kernel_width=0), E.KDA_ERR_SHAPE),
                     (dict(kernel_width=9), E.KDA_ERR_SHAPE), (dict(total=7), E.KDA_ERR_SHAPE), (dict(max_t=65, total=130), E.KDA_ERR_SHAPE),
                     (dict(x=None), E.KDA_ERR_NULL), (dict(conv_slot=None), E.KDA_ERR_NULL), (dict(y=P + 1), E.KDA_ERR_ALIGN),
                     (dict(bias=P + 2), E.KDA_ERR_ALIGN)):
        assert call(make(ConvWindowDesc, WIN), make(ConvArgs, CONV, **kw), P, P, None) == code, kw
    assert call(make(ConvWindowDesc, WIN), make(ConvArgs, CONV), None, P, None) == E.KDA_ERR_NULL
    assert call(make(ConvWindowDesc, WIN), make(ConvArgs, CONV), P, P, None, kda.KDA_LAUNCH_PDL_EARLY_STATE) == E.KDA_ERR_ARG
    assert call(make(ConvWindowDesc, WIN), make(ConvArgs, CONV, n=0, total=0), None, None, None) == E.KDA_OK


def test_accept_refusals(lib):
    call = lib.kda_accept_raw
    for kw, code in ((dict(n=-1), E.KDA_ERR_ARG), (dict(reserved=3), E.KDA_ERR_ARG), (dict(dtype=3), E.KDA_ERR_DTYPE_UNSUPPORTED),
                     (dict(vocab=0), E.KDA_ERR_SHAPE), (dict(vocab=(1 << 30) + 1, p_stride=1 << 31, q_stride=1 << 31), E.KDA_ERR_SHAPE),
                     (dict(p_stride=99), E.KDA_ERR_SHAPE), (dict(q_stride=99), E.KDA_ERR_SHAPE), (dict(total=7), E.KDA_ERR_SHAPE),
                     (dict(max_t=65, total=130), E.KDA_ERR_SHAPE), (dict(n=1 << 29, max_t=0, total=0), E.KDA_ERR_SHAPE),
                     (dict(p=None), E.KDA_ERR_NULL), (dict(tokens=None), E.KDA_ERR_NULL), (dict(u_last=None), E.KDA_ERR_NULL),
                     (dict(path=None), E.KDA_ERR_NULL), (dict(node=None), E.KDA_ERR_NULL), (dict(p=P + 2), E.KDA_ERR_ALIGN),
                     (dict(q=P + 1), E.KDA_ERR_ALIGN), (dict(tree=P + 4), E.KDA_ERR_ALIGN), (dict(token=P + 2), E.KDA_ERR_ALIGN)):
        assert call(make(AcceptArgs, ACCEPT, **kw), P, None) == code, kw
    assert call(make(AcceptArgs, ACCEPT), None, None) == E.KDA_ERR_NULL
    assert call(make(AcceptArgs, ACCEPT), P, None, kda.KDA_LAUNCH_PDL_EARLY_STATE) == E.KDA_ERR_ARG
    assert call(make(AcceptArgs, ACCEPT, n=0, total=0), None, None) == E.KDA_OK
    assert call(make(AcceptArgs, ACCEPT, max_t=0, total=0), None, None) == E.KDA_OK
    assert lib.lib.kda_accept(None, P, 0, None) == E.KDA_ERR_NULL


def test_kv4_tree_refusals(lib):
    from kda_linear_attention_gated_gb300 import _build  # noqa: F401
    for fn, args in ((lib.lib.kda_kv4_append_tree, append_args), (lib.lib.kda_kv4_attend_tree, attend_args)):
        def call(tree, c=None, status=P, flags=0, fn=fn, args=args, **kw):
            return fn(ctypes.byref(c or cache_desc()), ctypes.byref(args(**kw)), tree, status, flags, None)
        assert call(None) == E.KDA_ERR_NULL
        assert call(P + 4) == E.KDA_ERR_ALIGN
        assert call(P, status=None) == E.KDA_ERR_NULL
        assert call(P, max_t=65, total=195) == E.KDA_ERR_SHAPE
        assert call(P, c=cache_desc(dim=96)) == E.KDA_ERR_SHAPE
        assert call(P, dtype=9) == E.KDA_ERR_DTYPE_UNSUPPORTED
        assert call(P, rope_rows=0) == E.KDA_ERR_SHAPE
        assert call(P, flags=kda.KDA_LAUNCH_PDL_EARLY_STATE) == E.KDA_ERR_ARG
        assert call(None, n=0, total=0) == E.KDA_OK
    for small in (0, kda.KDA_KV4_WORKSPACE_BYTES, kda.KDA_KV4_TREE_WORKSPACE_BYTES - 1):
        args = attend_args(workspace_bytes=small)
        assert lib.lib.kda_kv4_attend_tree(ctypes.byref(cache_desc()), ctypes.byref(args), P, P, 0, None) == E.KDA_ERR_SHAPE


def test_kv4_tree_tables_next_to_2_31_tokens_are_refused(lib):
    """The end of the last unit of 64 keys stays below 2^31."""
    one = cache_desc(heads=1, page_tokens=16)
    args = attend_args(table_cols=(2 ** 31 - 48) // 16, h_q=1, rot_dim=0, n=0, total=0)
    assert lib.lib.kda_kv4_attend_tree(ctypes.byref(one), ctypes.byref(args), P, P, 0, None) == E.KDA_ERR_SHAPE


def test_cpu_tensors_and_missing_trees_are_refused(lib):
    z = torch.zeros
    i32 = dict(dtype=torch.int32)
    st = z(1, **i32)
    with pytest.raises(ValueError):
        lib.kda_accept(z(3, 5), z(3, **i32), z(3), z(1), z(1, **i32), z(1, **i32), z(1, 3, **i32), z(1, **i32), st)
    with pytest.raises(ValueError):
        lib.kda_step_tree(z(4, 1, 16, 16), z(1, 2, **i32), z(2, 1, 16), z(2, 1, 16), z(2, 1, 16), z(2, 1, 16), z(2, 1),
                          z(2, dtype=torch.int64), z(2, 1, 16), st)
    with pytest.raises(ValueError):
        lib.kda_conv_step_tree(z(2, 3, 8), z(1, **i32), z(2, 8), z(8, 4), z(2, dtype=torch.int64), z(2, 8), st)
    pages = z(4, 2, 1, 18 * 64, dtype=torch.uint8)
    for call in (lambda: lib.kda_kv4_append_tree(pages, z(3, 2, **i32), z(3, **i32), z(3, 2, 64), z(3, 2, 64), None, st),
                 lambda: lib.kda_kv4_attend_tree(pages, z(3, 2, **i32), z(3, **i32), z(3, 4, 64), None, z(3, 4, 64), z(8), st)):
        with pytest.raises(ValueError, match="tree is required"):
            call()


# -- the references ------------------------------------------------------------
def test_reference_step_on_a_chain_is_the_recurrence(oracle_mod):
    """A chain's states and outputs against the oracle's speculative verify."""
    import numpy as np
    g = torch.Generator().manual_seed(3)
    t, hv, kd, vd = 5, 2, 32, 16
    q, k, a = (torch.randn(t, hv, kd, generator=g) for _ in range(3))
    v, b = torch.randn(t, hv, vd, generator=g), torch.randn(t, hv, generator=g)
    pool = 0.1 * torch.randn(t + 1, hv, kd, vd, generator=g)
    o, eo, S, es = ref.step(pool[0], ref.parents(t, "chain"), q, k, v, a, b)
    got = pool.numpy().copy()
    o2 = oracle_mod.spec_verify(got, np.array([0], dtype=np.int32), np.arange(1, t + 1, dtype=np.int32)[None], q[None], k[None], v[None],
                                a[None], b[None])
    assert np.abs(o.numpy() - np.asarray(o2)[0]).max() < 1e-7
    assert np.abs(S.numpy() - got[1:]).max() < 1e-7
    assert eo.max() < 1e-3 and es.max() < 1e-3 and eo.min() > 0


def test_reference_acceptance_gives_the_targets_distribution():
    """Drafts drawn from q (two siblings) or given, and then accepted or redrawn: the first token's distribution is p's.

    200,000 trials a case; each frequency within 6 standard deviations (of at most sqrt(p (1 - p) / N))."""
    g = torch.Generator().manual_seed(11)
    vocab, trials = 5, 200_000
    p = torch.softmax(torch.randn(vocab, generator=g), 0).double()
    q = torch.softmax(torch.randn(vocab, generator=g), 0).double()
    for drawn in (True, False):
        x = torch.multinomial(q, 2 * trials, replacement=True, generator=g).view(trials, 2) if drawn else torch.tensor([[1, 3]]).expand(trials, 2)
        u = torch.rand(trials, 3, generator=g).double()
        # all trials at once, the same steps as accept() of _tree_ref
        w, z = p.expand(trials, vocab).clone(), torch.ones(trials).double()
        token = torch.full((trials,), -1)
        for i in range(2):
            xi = x[:, i:i + 1]
            held = w.gather(1, xi).squeeze(1)
            yes = (token < 0) & (u[:, i] * (q[xi.squeeze(1)] if drawn else 1.0) * z < held)
            token = torch.where(yes, xi.squeeze(1), token)
            left = (w - z[:, None] * q).clamp(min=0) if drawn else w.scatter(1, xi, 0.0)
            w, z = left, left.sum(1) if drawn else z - held
        cum = w.cumsum(1)
        redrawn = (cum <= u[:, 2:] * cum[:, -1:]).sum(1).clamp(max=vocab - 1)
        token = torch.where(token < 0, redrawn, token)
        f = torch.bincount(token, minlength=vocab).double() / trials
        assert ((f - p).abs() <= 6 * (p * (1 - p) / trials).sqrt()).all(), drawn
        for s in range(40):      # and accept() takes those steps
            rows = p.expand(3, vocab), q.expand(3, vocab) if drawn else None
            path, nxt = ref.accept(rows[0], rows[1], [0, int(x[s, 0]), int(x[s, 1])], [-1, 0, 0], [0.0, u[s, 0], u[s, 1]], u[s, 2])
            first = int(x[s, path[1] - 1]) if len(path) > 1 else nxt
            assert first == int(token[s])
