"""The operators around the recurrence launch on the current device: tensors that
live on another one are refused before anything is launched."""
import pytest
import torch

import kda_linear_attention_gated_gb300 as kda


class Elsewhere(torch.Tensor):
    """A tensor that says it lives on the next GPU."""

    def get_device(self):
        return torch.Tensor.get_device(self) + 1


@pytest.fixture(scope="module")
def lib(built_libs):
    return kda.KdaLibrary(torch.float32)


def calls():
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    i32, u8 = torch.int32, torch.uint8
    pages, table, ctx, st, cu = z(4, 2, 1, 18 * 64, d=u8), z(3, 2, d=i32), z(3, d=i32), z(1, d=i32), torch.arange(4, dtype=i32, device="cuda")
    rope = dict(cos=z(32, 32), sin=z(32, 32), cu_seqlens=cu)
    return {"kda_kv4_append": (dict(pages=pages, page_table=table, ctx_len=ctx, k=z(3, 2, 64), v=z(3, 2, 64), status=st, k_out=z(3, 2, 64),
                                    v_out=z(3, 2, 64), **rope), dict(max_t=1)),
            "kda_kv4_attend": (dict(pages=pages, page_table=table, ctx_len=ctx, q=z(3, 4, 64), o=z(3, 4, 64),
                                    workspace=z(kda.KDA_KV4_WORKSPACE_BYTES, d=u8), status=st, **rope), dict(max_t=1)),
            "kda_head_norm": (dict(o=z(3, 2, 64), weight=z(64), y=z(3, 2, 64), gate=z(3, 2, 64)), {}),
            "kda_block_norm": (dict(residual=z(3, 64), y=z(3, 64), residual_out=z(3, 64), w_post=z(64), gate=z(3, 64), scale=z(64), w_pre=z(64),
                                    x=z(3, 64)), {})}


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["kda_kv4_append", "kda_kv4_attend", "kda_head_norm", "kda_block_norm"])
def test_each_tensor_on_another_gpu_is_refused(lib, name):
    tensors, rest = calls()[name]
    call = getattr(lib, name)
    call(**tensors, **rest)
    for key, t in tensors.items():
        with pytest.raises(ValueError, match="cuda:"):
            call(**{**tensors, key: t.as_subclass(Elsewhere)}, **rest)
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["kda_kv4_append", "kda_kv4_attend", "kda_head_norm", "kda_block_norm"])
def test_tensors_on_another_gpu_than_the_current_one_are_refused(lib, name, monkeypatch):
    tensors, rest = calls()[name]
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        getattr(lib, name)(**tensors, **rest)
