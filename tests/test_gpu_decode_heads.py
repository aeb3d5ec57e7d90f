"""Decode over coded caches, query heads of one kv head that have nothing to do
with each other: one that is not finite, or larger by many powers of two, is no
matter of the others."""
import pytest
import torch

import paged_kv_cache_num_gb300 as pkv
from tests import prompt_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")


@pytest.mark.parametrize("dtype,bad", [(torch.bfloat16, INF), (torch.bfloat16, -INF), (torch.bfloat16, float("nan")), (torch.bfloat16, 2.0 ** 60),
                                       (torch.bfloat16, 2.0 ** 120), (torch.float16, INF), (torch.float16, float("nan")), (torch.float16, 2.0 ** 13)])
@pytest.mark.parametrize("kind,G,H,D,BS,scales,layout", [
    ("e4m3", 4, 4, 128, 32, "head", "flash"), ("e5m2", 8, 2, 64, 16, "head", "flash"), ("e4m3", 16, 2, 128, 32, "token", "flash"),
    ("i8", 8, 2, 128, 32, "block", "flash"), ("i8", 12, 1, 128, 16, "head", "flash"), ("i8", 4, 4, 128, 32, "head", "xvec"),
    ("u3", 4, 4, 128, 16, "head", "flash"), ("u3", 1, 8, 128, 32, "head", "flash"), ("u3", 1, 4, 128, 16, "head", "flash"), ("u3", 16, 2, 128, 32, "head", "flash")])
def test_one_head_apart(kind, G, H, D, BS, scales, layout, dtype, bad):
    ctx = [21, 300, 70]
    bt, P = R.tables(ctx, BS, seed=G)
    cache, kv, vv = R.make_cache(pkv, kind, P, BS, H, D, scales=scales, layout=layout, seed=G)
    g = torch.Generator().manual_seed(3)
    clean = torch.randn((len(ctx), G * H, D), generator=g).to(dtype)
    apart = sorted({0, G * H - 1})
    q = clean.clone()
    for h in apart:
        if abs(bad) == INF or bad != bad:
            q[:, h, 5] = bad
        else:
            q[:, h] *= bad
    rest = [h for h in range(G * H) if h not in apart]
    ref, mean, top, keys = (t[:, rest] if t.dim() > 1 else t for t in R.prefill(clean, kv, vv, bt, range(len(ctx) + 1), ctx, D ** -0.5))
    vmax = float(vv.abs().max())
    tol = R.prefill_tolerance(ref, mean, top, keys, vmax, dtype, D)
    # weights are f16 whatever the output's type; int8 codes are code + 1152 in the scores' products; 3-bit
    # codes are subnormals whose products are aligned as if they were 2^-14: a step each is 2^-23 of 1279
    # times |q|'s sum, 2^-13 of its largest element, times the scale, D / 16 + 2 of them, in the weight and in the sum;
    # 3-bit sums over the keys hold sums of codes up to 14 steps apart, half vmax each key
    step = 0.0
    if kind == "i8":
        step = 2.0 ** -23 * 1279 * float(clean.double().abs().sum(-1).max()) * float(kv.abs().max()) / 127 * (2 if scales == "block" else 1)
    if kind == "u3":
        step = 2.0 ** -13 * float(clean.abs().max()) * 0.75
        tol = tol + 2 * vmax * (keys[:, None, None] / 16 + 8) * 2.0 ** -23
    tol = tol + 2 * (D / 16 + 2) * step * D ** -0.5 * mean + 2.0 ** -11 * mean
    cl = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    for splits in (0, 1):
        out = pkv.paged_decode(q.to(DEV), cache, bt.to(DEV), cl, num_splits=splits).double().cpu()[:, rest]
        worst = float(((out - ref).abs() / tol).max())
        assert bool(torch.isfinite(out).all()) and worst <= 1.0, "%.3g of the tolerance, splits %d" % (worst, splits)


@pytest.mark.parametrize("kind,G", [("e4m3", 4), ("i8", 12), ("u3", 4), ("u3", 1), ("u3", 16)])
@pytest.mark.parametrize("big", [2.0 ** 100, 2.0 ** 122])
def test_heads_of_the_types_largest(kind, G, big):
    """Scores of ordinary size from queries at the upper end of bf16's range."""
    H, D, BS, ctx = 2, 128, 32, [90, 20]
    bt, P = R.tables(ctx, BS)
    cache, kv, vv = R.make_cache(pkv, kind, P, BS, H, D)
    base = torch.randn((2, G * H, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    cl = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    want = pkv.paged_decode(base.to(DEV), cache, bt.to(DEV), cl, sm_scale=0.125, num_splits=1)
    got = pkv.paged_decode((base * big).to(DEV), cache, bt.to(DEV), cl, sm_scale=0.125 / big)
    # the same scores: outputs up to 4 that differ by the roundings of two kernels, half a step each and the weights'
    assert float((got.double() - want.double()).abs().max()) <= 2 * 2.0 ** -8 * float(want.abs().max()) + 0.01
