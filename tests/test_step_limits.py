"""The batch limits of extend_tables and trim_tables, each with arguments that are
right otherwise.  CPU only: the pointers are made up."""
import ctypes

import pytest

from tests.test_abi import _fake

SHAPE, UNSUPPORTED = -3, -5
by = ctypes.byref


@pytest.fixture(scope="module")
def m():
    from paged_kv_cache_num_gb300 import build
    build.build()
    from paged_kv_cache_num_gb300 import pkv
    pkv.lib()
    return pkv


def args(m, B, out=None):
    f = _fake
    return [by(x) for x in (f((B, 5), m.I32), f((B,), m.I32), f((B,), m.I32), f((40,), m.I32), f((1,), m.I32))], by(f((out or B,), m.I32)), by(f((1,), m.I32))


def test_trim(m):
    for B, want in ((16385, UNSUPPORTED), (1 << 20, UNSUPPORTED)):
        first, out, left = args(m, B)
        assert m.lib().pkv_trim_tables(*first, 16, out, left, None, None) == want
    first, out, left = args(m, 16385, out=16384)
    assert m.lib().pkv_trim_tables(*first, 16, out, left, None, None) == SHAPE


def test_extend(m):
    first, out, left = args(m, 16385)
    rows = [by(_fake((64,), t)) for t in (m.I32, m.I32, m.I64)]
    assert m.lib().pkv_extend_tables(*first, 16, out, by(_fake((16386,), m.I32)), *rows, left, None, None) == UNSUPPORTED
