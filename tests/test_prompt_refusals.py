"""What paged_prefill, kv_append_dynamic and kv_gather refuse, before any
launch.  CPU only: the pointers are made up, and every call ends in the
argument checks."""
import ctypes

import pytest
import torch

from tests.test_abi import _cache, _fake

NULL, DTYPE, SHAPE, LAYOUT, UNSUPPORTED, WORKSPACE, VALUE = -1, -2, -3, -4, -5, -6, -7


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_num_gb300 import build
    build.build()
    from paged_kv_cache_num_gb300 import pkv
    return pkv.lib()


@pytest.fixture(scope="module")
def m():
    from paged_kv_cache_num_gb300 import pkv
    return pkv


by = ctypes.byref


def granular(m, kind, mode, P=4, BS=16, H=2, D=64):
    c = _cache(kind, P, BS, H, D)
    c.scale_mode = mode
    c.k_scales = _fake((P, H) if mode == 1 else (P, BS, H), m.F32)
    c.v_scales = _fake((P, H) if mode == 1 else (P, BS, H), m.F32, ptr=0x30000)
    return c


def prefill(lib, m, cache=None, q=None, bt=None, st=None, cl=None, out=None, scale=0.1, ws=None, wsn=0):
    T, Hq, D = 6, 4, 64
    cache = cache or _cache(m.F16, D=D)
    q = q or _fake((T, Hq, D), m.F16)
    return lib.pkv_paged_prefill(by(q), by(cache), by(bt or _fake((2, 5), m.I32)), by(st or _fake((3,), m.I32)),
                                 by(cl or _fake((2,), m.I32)), ctypes.c_float(scale),
                                 by(out or _fake((T, Hq, D), m.F16)), ws, wsn, None, None)


def test_prefill_refusals(lib, m):
    T, Hq, D = 6, 4, 64
    f = _fake
    assert prefill(lib, m, q=f((T, Hq, D), m.F32)) == DTYPE
    assert prefill(lib, m, q=f((T, Hq, D), m.BF16)) == DTYPE              # a 16-bit cache of the other type
    assert prefill(lib, m, q=f((T, 3, D), m.F16)) == SHAPE                # 3 q heads over 2 kv heads
    assert prefill(lib, m, q=f((T, 0, D), m.F16)) == SHAPE
    assert prefill(lib, m, q=f((T, Hq, 128), m.F16)) == SHAPE
    assert prefill(lib, m, q=f((T, Hq), m.F16)) == SHAPE
    assert prefill(lib, m, q=f((T, Hq, D), m.F16, (Hq * D * 2, D * 2, 2))) == LAYOUT
    assert prefill(lib, m, q=f((T, Hq, D), m.F16, ptr=0x10008)) == LAYOUT
    assert prefill(lib, m, q=f((T, Hq, D), m.F16, (Hq * D + 4, D, 1))) == LAYOUT
    assert prefill(lib, m, cache=_cache(m.F16, D=96), q=f((T, Hq, 96), m.F16)) == UNSUPPORTED
    assert prefill(lib, m, cache=_cache(m.F16, BS=4)) == UNSUPPORTED
    assert prefill(lib, m, cache=_cache(m.F16, BS=48)) == UNSUPPORTED
    assert prefill(lib, m, cache=_cache(m.F16, BS=512)) == UNSUPPORTED
    assert prefill(lib, m, cache=_cache(m.E4M3)) == NULL                  # no scales
    assert prefill(lib, m, bt=f((2, 5), m.I64)) == DTYPE
    assert prefill(lib, m, bt=f((2,), m.I32)) == SHAPE
    assert prefill(lib, m, st=f((2,), m.I32)) == SHAPE                    # batch entries, not batch + 1
    assert prefill(lib, m, st=f((3,), m.I64)) == DTYPE
    assert prefill(lib, m, cl=f((3,), m.I32)) == SHAPE
    assert prefill(lib, m, cl=f((2,), m.I64)) == DTYPE
    assert prefill(lib, m, out=f((T, Hq, D), m.BF16)) == DTYPE
    assert prefill(lib, m, out=f((T + 1, Hq, D), m.F16)) == SHAPE
    assert prefill(lib, m, out=f((T, Hq, D), m.F16, (Hq * D * 2, D * 2, 2))) == LAYOUT
    for bad in (float("nan"), float("inf")):
        assert prefill(lib, m, scale=bad) == VALUE
    assert prefill(lib, m, q=f((1 << 30, Hq, D), m.F16)) == UNSUPPORTED   # 2^31 rows of a kv head
    assert prefill(lib, m, bt=f((1 << 20, 5), m.I32)) == UNSUPPORTED
    assert prefill(lib, m, bt=f((2, 1 << 27), m.I32)) == UNSUPPORTED      # rows of 2^31 tokens
    n = ctypes.c_size_t(0)
    assert lib.pkv_paged_prefill_workspace(by(f((T, Hq, D), m.F16)), by(_cache(m.F16)), by(f((2, 5), m.I32)), None) == NULL
    assert lib.pkv_paged_prefill_workspace(by(f((T, Hq, D), m.F32)), by(_cache(m.F16)), by(f((2, 5), m.I32)), by(n)) == DTYPE
    assert lib.pkv_paged_prefill_launches(by(f((T, Hq, D), m.F16)), by(_cache(m.F16)), by(f((2, 5), m.I32)), None) == NULL


def test_prefill_without_work(lib, m):
    """No tokens, or no sequences: nothing to launch."""
    assert prefill(lib, m, q=_fake((0, 4, 64), m.F16, ptr=0), out=_fake((0, 4, 64), m.F16, ptr=0), ws=0x10000, wsn=1 << 40) == 0
    assert prefill(lib, m, bt=_fake((0, 5), m.I32, ptr=0), st=_fake((1,), m.I32), cl=_fake((0,), m.I32, ptr=0),
                   ws=0x10000, wsn=1 << 40) == 0


def test_dynamic_append_refusals(lib, m):
    T, H, D = 3, 2, 64

    def go(cache, kn=None, sm=None):
        kn = kn or _fake((T, H, D), m.F16)
        return lib.pkv_kv_append_dynamic(by(kn), by(kn), by(sm or _fake((T,), m.I64)), by(cache), None, None)

    assert go(_cache(m.F16)) == VALUE                                     # no per-token scales
    assert go(granular(m, m.E4M3, 1)) == VALUE
    assert go(granular(m, m.F16, 2)) == UNSUPPORTED
    assert go(granular(m, m.E4M3, 2, D=96), kn=_fake((T, H, 96), m.F16)) == UNSUPPORTED
    c = granular(m, m.E4M3, 2)
    assert go(c, sm=_fake((T,), m.I32)) == DTYPE
    assert go(c, sm=_fake((T + 1,), m.I64)) == SHAPE
    assert go(c, kn=_fake((T, H, D), m.F32)) == DTYPE
    assert go(c, kn=_fake((T, 3, D), m.F16)) == SHAPE
    assert go(c, kn=_fake((T, H, 128), m.F16)) == SHAPE
    assert go(c, kn=_fake((T, H, D), m.F16, (2 * H * D, 2 * D, 2))) == LAYOUT
    c.k_scales.dtype = m.F16
    assert go(c) == DTYPE
    assert lib.pkv_kv_append_dynamic(by(_fake((T, H, D), m.F16)), None, by(_fake((T,), m.I64)),
                                     by(granular(m, m.E4M3, 2)), None, None) == NULL
    assert lib.pkv_kv_append_dynamic(by(_fake((T, H, D), m.F16)), by(_fake((T, H, D), m.F16)),
                                     by(_fake((T,), m.I64)), None, None, None) == NULL
    # the plain append still refuses a per-token cache
    kn = _fake((T, H, D), m.F16)
    assert lib.pkv_kv_append(by(kn), by(kn), by(_fake((T,), m.I64)), by(granular(m, m.E4M3, 2)), None, None) == UNSUPPORTED


def test_gather_refusals(lib, m):
    T, H, D = 3, 2, 64

    def go(cache, ko=None, vo=None, sm=None):
        ko = ko or _fake((T, H, D), m.F16)
        return lib.pkv_kv_gather(by(cache), by(sm or _fake((T,), m.I64)), by(ko), by(vo or ko), None, None)

    c = _cache(m.F16)
    assert go(c, sm=_fake((T,), m.I32)) == DTYPE
    assert go(c, sm=_fake((T, 1), m.I64)) == SHAPE
    assert go(c, ko=_fake((T, H, D), m.F32)) == DTYPE
    assert go(c, ko=_fake((T, H, D), m.F16), vo=_fake((T, H, D), m.BF16)) == DTYPE
    assert go(c, ko=_fake((T + 1, H, D), m.F16)) == SHAPE
    assert go(c, ko=_fake((T, 3, D), m.F16)) == SHAPE
    assert go(c, vo=_fake((T, H, 128), m.F16)) == SHAPE
    assert go(c, ko=_fake((T, H, D), m.F16, (2 * H * D, 2 * D, 2))) == LAYOUT
    assert go(_cache(m.E4M3)) == NULL
    assert go(_cache(m.F16, D=60), ko=_fake((T, H, 60), m.F16)) in (LAYOUT, UNSUPPORTED)
    assert go(_cache(m.F16, D=24), ko=_fake((0, H, 24), m.F16, ptr=0), sm=_fake((0,), m.I64, ptr=0)) == 0
    assert lib.pkv_kv_gather(None, by(_fake((T,), m.I64)), by(_fake((T, H, D), m.F16)), by(_fake((T, H, D), m.F16)),
                             None, None) == NULL


def test_python_refusals(m):
    """CPU tensors are refused by name."""
    import paged_kv_cache_num_gb300 as pkv
    k = torch.zeros((4, 16, 2, 64), dtype=torch.float16)
    c = pkv.KVCache("f16", k, k)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_prefill(torch.zeros((3, 4, 64), dtype=torch.float16), c, torch.zeros((1, 4), dtype=torch.int32), i, i[:1])
    with pytest.raises(ValueError, match="CUDA"):
        pkv.kv_gather(c, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.kv_append_dynamic(k[0], k[0], torch.zeros(16, dtype=torch.int64), c)


class _Fake:
    """Stands for a tensor or stream of a CUDA device that this machine has not."""

    def __init__(self, dev):
        self.device_index = dev

    def get_device(self):
        return self.device_index


def test_mixed_devices_are_refused(m):
    with pytest.raises(ValueError, match="one device"):
        m._one_device(_Fake(0), None, _Fake(1))
    with pytest.raises(ValueError, match="the stream is on"):
        m._elsewhere(0, _Fake(1))
    assert m._one_device(_Fake(1), None, _Fake(1)) == 1


def test_more_than_four_dims_are_refused(m):
    with pytest.raises(ValueError, match="dims"):
        m._desc(torch.zeros((1, 1, 1, 1, 1), dtype=torch.float16))
