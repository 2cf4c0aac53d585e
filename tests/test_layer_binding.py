"""The binding of the operators around the recurrence: packed argument structs
match the ctypes mirrors of the C structs, and bad tensors are refused in Python
before the library is called (no GPU)."""
import ctypes

import pytest
import torch

import kda_linear_attention_gated_gb300 as kda

PAIRS = [(kda._PACK_KV4_CACHE, kda.Kv4CacheDesc), (kda._PACK_KV4_APPEND, kda.Kv4AppendArgs), (kda._PACK_KV4_ATTEND, kda.Kv4AttendArgs),
         (kda._PACK_HEAD_NORM, kda.HeadNormArgs), (kda._PACK_BLOCK_NORM, kda.BlockNormArgs)]


@pytest.mark.parametrize("packer,mirror", PAIRS, ids=[m.__name__ for _, m in PAIRS])
def test_packed_arguments_have_the_structs_layout(packer, mirror):
    assert packer.size == ctypes.sizeof(mirror)
    values = [float(i + 1) if kind is ctypes.c_float else i + 1 for i, (_, kind) in enumerate(mirror._fields_)]
    got = mirror.from_buffer_copy(packer.pack(*values))
    assert [getattr(got, name) for name, _ in mirror._fields_] == values


@pytest.fixture(scope="module")
def lib(built_libs):
    return kda.KdaLibrary(torch.float32)


def test_cpu_tensors_and_wrong_shapes_are_refused(lib):
    t = torch.zeros
    with pytest.raises(ValueError):
        lib.kda_head_norm(t(2, 3, 16), t(16), t(2, 3, 16))                    # not on the GPU
    with pytest.raises(ValueError):
        lib.kda_block_norm(t(2, 16), None, None)                              # neither y nor x
    with pytest.raises(ValueError):
        lib.kda_block_norm(t(2, 16), t(2, 16), t(2, 16))
    pages = t(4, 2, 1, 18 * 64, dtype=torch.uint8)
    ids, st = t(3, 2, dtype=torch.int32), t(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        lib.kda_kv4_append(pages, ids, t(3, dtype=torch.int32), t(3, 2, 64), t(3, 2, 64), st)
    with pytest.raises(ValueError):
        lib.kda_kv4_attend(pages, ids, t(3, dtype=torch.int32), t(3, 4, 64), t(3, 4, 64), t(8), st)


@pytest.mark.gpu
def test_gpu_tensors_of_wrong_shape_type_or_stride_are_refused(lib):
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    i32, u8, bf = torch.int32, torch.uint8, torch.bfloat16
    pages, table, ctx, st = z(4, 2, 1, 18 * 64, d=u8), z(3, 2, d=i32), z(3, d=i32), z(1, d=i32)
    k, q, ws = z(3, 2, 64), z(3, 4, 64), z(kda.KDA_KV4_WORKSPACE_BYTES, d=u8)
    good = dict(pages=pages, page_table=table, ctx_len=ctx, k=k, v=k, status=st)
    lib.kda_kv4_append(**good)
    for bad in (dict(pages=pages.float()), dict(pages=pages[..., :1000]), dict(pages=pages.transpose(0, 1)), dict(ctx_len=z(2, d=i32)),
                dict(page_table=table.long()), dict(k=z(3, 3, 64)), dict(v=k.to(bf)), dict(k=z(3, 64, 2).transpose(1, 2)),
                dict(cos=z(8, 16)), dict(cos=z(8, 16), sin=z(8, 8)), dict(cu_seqlens=z(4, d=i32)), dict(cu_seqlens=z(3, d=i32), max_t=1),
                dict(k_out=z(3, 2, 32)), dict(k_out=z(3, 2, 64), v_out=z(3, 2, 64, d=bf)), dict(status=z(2, d=i32))):
        with pytest.raises(ValueError):
            lib.kda_kv4_append(**{**good, **bad})
    good = dict(pages=pages, page_table=table, ctx_len=ctx, q=q, o=z(3, 4, 64), workspace=ws, status=st)
    lib.kda_kv4_attend(**good)
    for bad in (dict(o=z(3, 4, 64, d=bf)), dict(q=z(3, 4, 32)), dict(workspace=torch.zeros(9)), dict(scale=0), dict(o=z(4, 3, 64).transpose(0, 1))):
        with pytest.raises(ValueError):
            lib.kda_kv4_attend(**{**good, **bad})
    for bad, code in ((dict(workspace=ws[:64]), kda.KDA_ERR_SHAPE), (dict(window=-1), kda.KDA_ERR_ARG), (dict(q=z(3, 3, 64), o=z(3, 3, 64)), kda.KDA_ERR_SHAPE)):
        with pytest.raises(kda.KdaError) as e:
            lib.kda_kv4_attend(**{**good, **bad})
        assert e.value.code == code
    with pytest.raises(ValueError):
        lib.kda_head_norm(q, z(64), q, gate=z(3, 64, 4).transpose(1, 2))
    with pytest.raises(kda.KdaError):
        lib.kda_head_norm(q, z(64), q, activation=5)
    with pytest.raises(ValueError):
        lib.kda_block_norm(z(3, 64), z(3, 64), z(3, 64), w_pre=z(63), x=z(3, 64))
    with pytest.raises(ValueError):
        lib.kda_block_norm(z(3, 64), z(3, 64), z(3, 64, d=bf))
    torch.cuda.synchronize()
    assert st.item() == 0
