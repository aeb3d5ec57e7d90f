"""Decode over blocks of every size that a cache may have, from one slot to 256."""
import pytest
import torch

import paged_kv_cache_num_gb300 as pkv
from tests import prompt_refs as R
from tests import u4_refs as U

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("BS", [1, 2, 4, 8, 128, 256])
@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3", "i8", "u3", "u4"])
def test_blocks(kind, BS):
    H, G, D = 2, 4, 64
    ctx = [1, BS, BS + 1, 3 * BS + 7, 300]
    bt, P = R.tables(ctx, BS, seed=BS)
    dtype = torch.bfloat16 if kind == "bf16" else torch.float16
    q = torch.randn((len(ctx), H * G, D), generator=torch.Generator().manual_seed(1)).to(dtype)
    cl = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    if kind == "u4":
        cache, vals, tops = U.make_cache(pkv, P, BS, H, D)
    else:
        cache, kv, vv = R.make_cache(pkv, kind, P, BS, H, D)
    for splits in (0, 1, 2):
        out = pkv.paged_decode(q.to(DEV), cache, bt.to(DEV), cl, num_splits=splits, err_flag=err)
        assert err.item() == 0
        if kind == "u4":
            U.close(out, U.decode_parts(q, vals, tops, bt, ctx, D ** -0.5), 4.5, dtype, D)
            continue
        ref = R.prefill(q, kv, vv, bt, range(len(ctx) + 1), ctx, D ** -0.5)
        tol = R.prefill_tolerance(*ref, float(vv.abs().max()), dtype, D)
        assert bool(((out.double().cpu() - ref[0]).abs() <= tol).all())
