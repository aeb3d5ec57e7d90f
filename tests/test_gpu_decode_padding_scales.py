"""paged_decode: scales of slots behind the contexts are no matter of any row."""
import pytest
import torch

from tests import scale_refs as S
from tests import prompt_refs as R

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("kind", ["e4m3", "e5m2", "i8"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("splits", [0, 2])
def test_scales_behind_the_context(kind, value, splits):
    import paged_kv_cache_num_gb300 as pkv
    H, G, D, BS, ctx = 4, 4, 128, 16, [5, 300, 1999]
    bt, P = R.tables(ctx, BS, seed=1)
    ks, vs = S.flat_scale(kind, (P, BS, H), 0.5), S.flat_scale(kind, (P, BS, H))
    cache, kv, vv = S.coded_cache(pkv, kind, "token", ks, vs, D, seed=2)
    q = torch.randn((len(ctx), H * G, D), generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    args = (bt.clamp(min=0).to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV))
    want = pkv.paged_decode(q, cache, *args, num_splits=splits)
    seen = torch.zeros((P, BS), dtype=torch.bool)
    for b, c in enumerate(ctx):
        for t in range(c):
            seen[bt[b, t // BS], t % BS] = True
    for t in (cache.k_scales, cache.v_scales):
        t[~seen.to(DEV)] = value
    assert torch.isfinite(want).all()
    assert torch.equal(pkv.paged_decode(q, cache, *args, num_splits=splits), want)
