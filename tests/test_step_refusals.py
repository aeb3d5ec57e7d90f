"""What norm_rope, norm_rope_append, extend_tables and trim_tables refuse, before
any launch.  CPU only: the pointers are made up."""
import ctypes

import pytest
import torch

from tests.test_abi import _cache, _fake

NULL, DTYPE, SHAPE, LAYOUT, UNSUPPORTED, VALUE = -1, -2, -3, -4, -5, -7
by = ctypes.byref


@pytest.fixture(scope="module")
def m():
    from paged_kv_cache_num_gb300 import build
    build.build()
    from paged_kv_cache_num_gb300 import pkv
    pkv.lib()
    return pkv


def ref(x):
    return None if x is None else by(x)


def shared(m, call):
    """Refusals that both forms of the norm and rotation share; call(**what differs)."""
    T, Hq, D = 3, 4, 64
    f = _fake
    assert call(q=f((T, Hq, D), m.F32)) == DTYPE
    assert call(q=f((T, Hq, D), m.BF16)) == DTYPE
    assert call(q=f((T + 1, Hq, D), m.F16)) == SHAPE
    assert call(q=f((T, Hq, 128), m.F16)) == SHAPE
    assert call(q=f((T, D), m.F16)) == SHAPE
    assert call(q=f((T, Hq, D), m.F16, (2 * Hq * D, 2 * D, 2))) == LAYOUT
    assert call(q_out=f((T, Hq, D), m.BF16)) == DTYPE
    assert call(q_out=f((T, Hq + 1, D), m.F16)) == SHAPE
    assert call(q_out=f((T, Hq, D), m.F16, (2 * Hq * D, 2 * D, 2))) == LAYOUT
    for n in ("qw", "kw"):
        assert call(**{n: f((D,), m.BF16)}) == DTYPE
        assert call(**{n: f((D // 2,), m.F16)}) == SHAPE
        assert call(**{n: f((D,), m.F16, (2,))}) == LAYOUT
        assert call(**{n: f((1, D), m.F16)}) == SHAPE
        assert call(**{n: f((D,), m.F16, ptr=0)}) == NULL
    assert call(qw=f((D,), m.F16), kw=f((D,), m.F32)) == DTYPE
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == VALUE
    assert call(cs=f((50, 64), m.F16)) == DTYPE
    assert call(cs=f((64,), m.F32)) == SHAPE
    for rot in (0, 8, 24, 80, 128):
        assert call(cs=f((50, rot), m.F32)) == UNSUPPORTED
    assert call(cs=f((50, 32), m.F32, (64, 2))) == LAYOUT
    assert call(cs=f((50, 32), m.F32, (34, 1))) == LAYOUT
    assert call(cs=f((50, 32), m.F32, ptr=0x10004)) == LAYOUT
    assert call(pos=f((T,), m.I64)) == DTYPE
    assert call(pos=f((T + 1,), m.I32)) == SHAPE


def test_norm_rope(m):
    T, Hq, H, D = 3, 4, 2, 64

    def call(q=None, k=None, qw=None, kw=None, eps=1e-6, cs=None, pos=None, q_out=None, k_out=None):
        return m.lib().pkv_norm_rope(ref(q or _fake((T, Hq, D), m.F16)), ref(k or _fake((T, H, D), m.F16)), ref(qw), ref(kw), eps,
                                     ref(cs or _fake((50, 32), m.F32)), ref(pos or _fake((T,), m.I32)), 0, ref(q_out or _fake((T, Hq, D), m.F16)),
                                     ref(k_out or _fake((T, H, D), m.F16)), None, None)

    shared(m, call)
    assert call(k=_fake((T, H, D), m.F32)) == DTYPE
    assert call(k=_fake((T, H, D), m.F16, (2 * H * D, 2 * D, 2))) == LAYOUT
    assert call(k_out=_fake((T, H, D), m.BF16)) == DTYPE
    assert call(k_out=_fake((T, H + 1, D), m.F16)) == SHAPE
    for d in (32, 96, 256):
        x = _fake((T, H, d), m.F16)
        assert call(q=x, k=x, q_out=x, k_out=x) == UNSUPPORTED
    none = _fake((0, H, D), m.F16, ptr=0)
    assert call(q=none, k=none, q_out=none, k_out=none, pos=_fake((0,), m.I32, ptr=0)) == 0
    assert m.lib().pkv_norm_rope(None, None, None, None, 0.0, None, None, 0, None, None, None, None) == NULL


def test_norm_rope_append(m):
    T, Hq, H, D = 3, 4, 2, 64

    def call(q=None, k=None, v=None, qw=None, kw=None, eps=1e-6, cs=None, pos=None, q_out=None, sm=None, cache=None):
        kv = _fake((T, H, D), m.F16)
        return m.lib().pkv_norm_rope_append(ref(q or _fake((T, Hq, D), m.F16)), ref(k or kv), ref(v or kv), ref(qw), ref(kw), eps,
                                            ref(cs or _fake((50, 32), m.F32)), ref(pos or _fake((T,), m.I32)), 0, ref(sm or _fake((T,), m.I64)),
                                            ref(cache or _cache(m.F16, H=H, D=D)), ref(q_out or _fake((T, Hq, D), m.F16)), None, None)

    shared(m, call)
    assert call(sm=_fake((T,), m.I32)) == DTYPE
    assert call(sm=_fake((T + 1,), m.I64)) == SHAPE
    assert call(cache=_cache(m.BF16, H=H, D=D)) == DTYPE
    assert call(cache=_cache(m.F16, H=3, D=D)) == SHAPE
    assert call(cache=_cache(m.E4M3, H=H, D=D)) == NULL                   # no scales
    assert call(v=_fake((T, H, D), m.BF16)) == DTYPE
    x = _fake((T, H, 96), m.F16)
    assert call(q=x, k=x, v=x, q_out=x, cache=_cache(m.F16, H=H, D=96)) == UNSUPPORTED
    kv = _fake((T, H, D), m.F16)
    assert m.lib().pkv_norm_rope_append(by(kv), by(kv), by(kv), None, None, 0.0, by(_fake((50, 32), m.F32)), by(_fake((T,), m.I32)), 0,
                                        by(_fake((T,), m.I64)), None, by(kv), None, None) == NULL


def test_tables(m):
    B, M, P, N = 3, 5, 40, 64
    f = _fake
    ok = {"bt": f((B, M), m.I32), "a": f((B,), m.I32), "b": f((B,), m.I32), "fb": f((P,), m.I32), "fc": f((1,), m.I32), "out": f((B,), m.I32),
          "fl": f((1,), m.I32)}
    rows = {"qs": f((B + 1,), m.I32), "req": f((N,), m.I32), "pos": f((N,), m.I32), "sm": f((N,), m.I64)}

    def extend(BS=16, **kw):
        a = {**ok, **rows, **kw}
        return m.lib().pkv_extend_tables(*(by(a[n]) for n in ("bt", "a", "b", "fb", "fc")), BS, *(by(a[n]) for n in ("out", "qs", "req", "pos", "sm", "fl")), None, None)

    def trim(BS=16, **kw):
        a = {**ok, **kw}
        return m.lib().pkv_trim_tables(*(by(a[n]) for n in ("bt", "a", "b", "fb", "fc")), BS, *(by(a[n]) for n in ("out", "fl")), None, None)

    for call in (extend, trim):
        for n in ok:
            shape = tuple(ok[n].shape[:ok[n].ndim])
            assert call(**{n: f(shape, m.I64)}) == DTYPE, n
            assert call(**{n: f(shape, m.I32, ptr=0)}) == NULL, n
            assert call(**{n: f(shape + (1,), m.I32)}) == SHAPE, n
        for n in ("a", "b", "out", "fc", "fl"):
            assert call(**{n: f((B + 1,), m.I32)}) == SHAPE
        assert call(fb=f((P,), m.I32, (2,))) == LAYOUT
        for bs in (0, -16, 12):
            assert call(bs) == VALUE
        assert call(bt=f((B, 1 << 27), m.I32)) == UNSUPPORTED
        big = {n: f((16385,), m.I32) for n in ("a", "b", "out")}
        assert call(bt=f((16385, M), m.I32), qs=f((16386,), m.I32), **big) == UNSUPPORTED if call is extend else True
    assert extend(qs=f((B,), m.I32)) == SHAPE
    assert extend(req=f((N + 1,), m.I32)) == SHAPE
    assert extend(sm=f((N,), m.I32)) == DTYPE
    assert extend(pos=f((N,), m.I64)) == DTYPE
    assert extend(sm=f((N,), m.I64, (2,))) == LAYOUT
    assert extend(qs=f((B + 1,), m.I32, (2,))) == LAYOUT


def test_python(m):
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros((2, 2, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        m.norm_rope(x, x, torch.zeros((4, 32)), i)
    with pytest.raises(ValueError, match="CUDA"):
        m.norm_rope_append(x, x, x, torch.zeros((4, 32)), i, i.long(), m.KVCache("f16", x[None], x[None]))
    with pytest.raises(ValueError, match="CUDA"):
        m.extend_tables(i[None], i, i, i, i[:1], 16, 4)
    with pytest.raises(ValueError, match="CUDA"):
        m.trim_tables(i[None], i, i, i, i[:1], 16)
