"""What the calls refuse of 4-bit caches, before any launch.  CPU only: the
pointers are made up."""
import ctypes

import pytest
import torch

from tests.test_abi import _fake

NULL, DTYPE, SHAPE, LAYOUT, UNSUPPORTED = -1, -2, -3, -4, -5
by = ctypes.byref


@pytest.fixture(scope="module")
def m():
    from paged_kv_cache_num_gb300 import build
    build.build()
    from paged_kv_cache_num_gb300 import pkv
    pkv.lib()
    return pkv


def cache(m, P=4, BS=16, H=2, D=64, row=None):
    c = m._Cache()
    row = D // 2 if row is None else row
    c.k_cache, c.v_cache = _fake((P, BS, H, row), m.U4), _fake((P, BS, H, row), m.U4, ptr=0x20000)
    c.k_qscale, c.v_qscale = _fake((P, BS, H), m.F16), _fake((P, BS, H), m.F16)
    c.k_qzero, c.v_qzero = _fake((P, BS, H), m.U8), _fake((P, BS, H), m.U8)
    return c


def decode(m, c, D=64, Hq=4, q=None):
    n = ctypes.c_size_t(0)
    return m.lib().pkv_paged_decode_workspace(by(q or _fake((2, Hq, D), m.F16)), by(c), by(_fake((2, 5), m.I32)), 0, by(n))


def test_decode(m):
    assert decode(m, cache(m)) == 0
    assert decode(m, cache(m, D=128), D=128) == 0
    assert decode(m, cache(m, D=96), D=96) == UNSUPPORTED
    assert decode(m, cache(m, BS=48)) == UNSUPPORTED
    assert decode(m, cache(m, BS=512)) == UNSUPPORTED
    assert decode(m, cache(m), D=128) == SHAPE
    assert decode(m, cache(m), Hq=3) == SHAPE
    assert decode(m, cache(m), Hq=34) == UNSUPPORTED                      # 17 q heads a kv head
    c = cache(m)
    c.chunk_stride = 16
    assert decode(m, c) == UNSUPPORTED
    c = cache(m)
    c.scale_mode = 2
    assert decode(m, c) == UNSUPPORTED
    for i in range(3):                                                    # rows off the 16-byte boundary
        c = cache(m)
        c.k_cache.stride[i] += 8
        c.v_cache.stride[i] += 8
        assert decode(m, c) == LAYOUT
    c = cache(m)
    c.v_cache.stride[0] += 16
    assert decode(m, c) == LAYOUT
    c = cache(m)
    c.k_cache.data = 0x10008
    assert decode(m, c) == LAYOUT


@pytest.mark.parametrize("name,dtype", [("k_qscale", "F32"), ("v_qscale", "BF16"), ("k_qzero", "I8"), ("v_qzero", "F16")])
def test_metadata(m, name, dtype):
    c = cache(m)
    setattr(c, name, _fake((4, 16, 2), getattr(m, dtype)))
    assert decode(m, c) == DTYPE
    c = cache(m)
    setattr(c, name, _fake((4, 15, 2), m.F16 if "scale" in name else m.U8, (32, 2, 1)))
    assert decode(m, c) == SHAPE
    c = cache(m)
    setattr(c, name, _fake((4, 16), m.F16 if "scale" in name else m.U8))
    assert decode(m, c) == SHAPE
    c = cache(m)
    setattr(c, name, _fake((4, 16, 2), m.F16 if "scale" in name else m.U8, ptr=0))
    assert decode(m, c) == NULL
    c = cache(m)
    setattr(c, name, _fake((4, 16, 2), m.F16 if "scale" in name else m.U8, (32, 1, 16)))    # K and V apart
    assert decode(m, c) == LAYOUT


def test_append_and_gather(m):
    T, H, D = 3, 2, 64

    def append(c, kn):
        return m.lib().pkv_kv_append(by(kn), by(kn), by(_fake((T,), m.I64)), by(c), None, None)

    assert append(cache(m), _fake((T, H, D), m.F32)) == DTYPE
    assert append(cache(m), _fake((T, H, 128), m.F16)) == SHAPE
    assert append(cache(m, D=96), _fake((T, H, 96), m.F16)) == UNSUPPORTED
    assert append(cache(m), _fake((T, H, D), m.F16, (2 * H * D, 2 * D, 2))) == LAYOUT
    k = by(_fake((T, H, D), m.F16))
    assert m.lib().pkv_kv_append_dynamic(k, k, by(_fake((T,), m.I64)), by(cache(m)), None, None) == -7
    g = _fake((T, H, 96), m.F16)
    assert m.lib().pkv_kv_gather(by(cache(m, D=96)), by(_fake((T,), m.I64)), by(g), by(g), None, None) == UNSUPPORTED


def test_binding(m):
    z, s, d = torch.zeros((3, 16, 4), dtype=torch.uint8), torch.zeros((3, 16, 4), dtype=torch.float16), torch.zeros((3, 16, 4, 32), dtype=torch.uint8)
    c = m.KVCache("u4", d, d, k_qscale=s, k_qzero=z, v_qscale=s, v_qzero=z)
    assert c.head_dim == 64
    c._struct()
    with pytest.raises(ValueError, match="k_qscale"):
        m.KVCache("u4", d, d, k_qscale=s.float(), k_qzero=z, v_qscale=s, v_qzero=z)._struct()
    with pytest.raises(ValueError, match="v_qzero"):
        m.KVCache("u4", d, d, k_qscale=s, k_qzero=z, v_qscale=s, v_qzero=z.int())._struct()
    with pytest.raises(ValueError, match="k_cache"):
        m.KVCache("u4", d.short(), d.short(), k_qscale=s, k_qzero=z, v_qscale=s, v_qzero=z)._struct()
    with pytest.raises(ValueError, match="xvec"):
        m.KVCache.allocate("u4", 3, 16, 4, 64, device="cpu", layout="xvec")
    a = m.KVCache.allocate("u4", 3, 16, 4, 128, device="cpu", fill=0)
    assert a.k_cache.shape == (3, 16, 4, 64) and a.k_qscale.shape == (3, 16, 4) and a.head_dim == 128


def test_definition_of_a_row():
    """Worked by hand: range with zero in it, half-integer quotients to even."""
    from tests import u4_refs as U
    x = torch.zeros(64)
    x[:4] = torch.tensor([15.0, 7.5, 6.5, 0.4])                           # s = 1, z = 0
    c, s, z = U.quantise(x.half())
    assert s == 1 and z == 0 and c[:5].tolist() == [15, 8, 6, 0, 0]
    x[:4] = torch.tensor([-5.0, 10.0, 2.5, -0.5])                         # s = 1, z = 5
    c, s, z = U.quantise(x.half())
    assert s == 1 and z == 5 and c[:5].tolist() == [0, 15, 7, 5, 5]
    c, s, z = U.quantise(torch.full((64,), 3.0).half())                   # equal numbers keep their value
    assert z == 0 and (c == 15).all() and abs(float(s) * 15 - 3) < 3 * 2.0 ** -11
    c, s, z = U.quantise(torch.zeros(64).half())
    assert s == 0 and z == 0 and (c == 0).all()
    assert U.pack4(torch.tensor([[1, 2, 15, 0]])).tolist() == [[0x21, 0x0F]]
