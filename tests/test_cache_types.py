"""KVCache refuses tensors that its descriptors would misstate.  CPU only."""
import pytest
import torch

import paged_kv_cache_num_gb300 as pkv

P, BS, H, D = 3, 16, 4, 64


def rows(dtype, row=D):
    return torch.zeros((P, BS, H, row), dtype=dtype)


def scales(dtype=torch.float32, shape=(P, BS, H)):
    return torch.ones(shape, dtype=dtype)


@pytest.mark.parametrize("kind,dtype", [("f16", torch.float32), ("bf16", torch.uint8), ("e4m3", torch.bfloat16), ("i8", torch.int32)])
def test_rows_of_another_width(kind, dtype):
    one = scales(shape=(H,))
    with pytest.raises(ValueError, match="k_cache"):
        pkv.KVCache(kind, rows(dtype), rows(dtype), k_scale=one, v_scale=one)._struct()


@pytest.mark.parametrize("mode,shape", [("token", (P, BS, H)), ("block", (P, H))])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float64])
def test_granular_scales_of_another_type(mode, shape, dtype):
    """kv_append_dynamic would write 32 bits to each."""
    c = pkv.KVCache("e4m3", rows(torch.uint8), rows(torch.uint8), scale_mode=mode, k_scales=scales(dtype, shape),
                    v_scales=scales(dtype, shape))
    with pytest.raises(ValueError, match="float32"):
        c._struct()


@pytest.mark.parametrize("bad", [torch.ones(H, dtype=torch.float64), torch.ones(1), torch.ones(1).expand(H), torch.ones(2 * H)[::2]])
def test_head_scales_that_are_no_row_of_floats(bad):
    with pytest.raises(ValueError, match="k_scale"):
        pkv.KVCache("i8", rows(torch.int8), rows(torch.int8), k_scale=bad, v_scale=torch.ones(H))._struct()


def test_three_bit_metadata_of_another_type():
    z = scales(torch.uint8)
    with pytest.raises(ValueError, match="k_qscale"):
        pkv.KVCache("u3", rows(torch.uint8, 24), rows(torch.uint8, 24), k_qscale=scales(), v_qscale=scales(), k_qzero=z, v_qzero=z)._struct()
    with pytest.raises(ValueError, match="k_qzero"):
        pkv.KVCache("u3", rows(torch.uint8, 24), rows(torch.uint8, 24), k_qscale=scales(torch.float16), v_qscale=scales(torch.float16),
                    k_qzero=scales(torch.int32), v_qzero=scales(torch.int32))._struct()


def test_right_types():
    one = scales(shape=(H,))
    for kind, dtype in (("f16", torch.float16), ("bf16", torch.bfloat16)):
        pkv.KVCache(kind, rows(dtype), rows(dtype))._struct()
    for kind, dtype in (("e4m3", torch.uint8), ("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2), ("i8", torch.int8)):
        pkv.KVCache(kind, rows(dtype), rows(dtype), k_scale=one, v_scale=one)._struct()
        pkv.KVCache(kind, rows(dtype), rows(dtype), scale_mode="token", k_scales=scales(), v_scales=scales())._struct()
    z, q = scales(torch.uint8), scales(torch.float16)
    pkv.KVCache("u3", rows(torch.uint8, 24), rows(torch.uint8, 24), k_qscale=q, v_qscale=q, k_qzero=z, v_qzero=z)._struct()
