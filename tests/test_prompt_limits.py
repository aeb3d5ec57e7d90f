"""Limits of paged_prefill's sizes, checked before any launch.  CPU only."""
import ctypes

import pytest

from tests.test_abi import _cache, _fake
from tests.test_prompt_refusals import UNSUPPORTED, lib, m  # noqa: F401


@pytest.mark.parametrize("BS", [8, 16, 128, 256])
def test_tokens_to_a_table_row(lib, m, BS):  # noqa: F811
    """Key tiles of 128 tokens are counted up from the context's length: it has
    to stay 256 below 2^31."""
    q, n = _fake((6, 4, 64), m.F16), ctypes.c_size_t(0)
    by = ctypes.byref
    for tokens, want in ((2 ** 31 - 256, 0), (2 ** 31 - 256 + BS, UNSUPPORTED), (2 ** 31 - BS, 0 if BS == 256 else UNSUPPORTED),
                         (2 ** 31, UNSUPPORTED)):
        bt = _fake((2, tokens // BS), m.I32)
        assert lib.pkv_paged_prefill_workspace(by(q), by(_cache(m.F16, BS=BS)), by(bt), by(n)) == want
