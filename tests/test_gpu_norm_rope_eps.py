"""norm_rope with eps = 0: rows whose mean square is a normal fp32 number follow the
formula; the others have no quotient in fp32, and are no matter of their neighbours."""
import pytest
import torch

import paged_kv_cache_num_gb300 as pkv
from tests.test_gpu_norm_rope import DEV, check, rand, table, turned

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype,amps", [(torch.float16, (1.0, 2.0 ** -9, 2.0 ** 11)), (torch.bfloat16, (1.0, 2.0 ** -55, 2.0 ** 55))])
@pytest.mark.parametrize("D", [64, 128])
def test_no_eps(D, dtype, amps, pairs):
    x = torch.cat([rand((9, 3, D), i) * a for i, a in enumerate(amps)]).to(dtype)
    w, cs = rand((D,), 7), table(D)
    pos = torch.arange(x.shape[0], dtype=torch.int32) * 31
    q, k = pkv.norm_rope(x.to(DEV), x.to(DEV), cs.to(DEV), pos.to(DEV), w.to(DEV), w.to(DEV), eps=0.0, interleaved=pairs)
    check(q, *turned(x, w, cs, pos, 0.0, pairs), dtype, D)
    assert torch.equal(q, k)


def test_rows_without_a_mean():
    """A row of zeros has none; nor, in fp32, has one whose squares are below its range."""
    x = rand((4, 2, 128), 1, torch.bfloat16)
    x[1, 0] = 0
    x[2, 1] *= 1e-30
    cs, pos, w = table(128), torch.arange(4, dtype=torch.int32), torch.ones(128)
    q = pkv.norm_rope(x.to(DEV), x.to(DEV), cs.to(DEV), pos.to(DEV), w.to(DEV), w.to(DEV), eps=0.0)[0].cpu()
    assert q[1, 0].isnan().all() and not torch.isfinite(q[2, 1]).any()
    want, big = turned(x, w, cs, pos, 0.0, False)
    for t, h in ((0, 0), (0, 1), (1, 1), (2, 0), (3, 0), (3, 1)):
        check(q[t, h], want[t, h], big[t, h], torch.bfloat16, 128)
    # with an eps they are what the formula gives
    q = pkv.norm_rope(x.to(DEV), x.to(DEV), cs.to(DEV), pos.to(DEV), w.to(DEV), w.to(DEV), eps=1e-12)[0]
    check(q, *turned(x, w, cs, pos, 1e-12, False), torch.bfloat16, 128)
