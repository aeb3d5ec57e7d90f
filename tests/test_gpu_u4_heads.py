"""Decode over 4-bit caches, query heads of one kv head that have nothing to do
with each other: one that is not finite, or larger by many powers of two, is no
matter of the others."""
import pytest
import torch

import paged_kv_cache_num_gb300 as pkv
from tests import prompt_refs as R
from tests import u4_refs as U
from tests.test_gpu_u4 import DEV, rand

pytestmark = pytest.mark.gpu

INF = float("inf")


def spoil(q, heads, bad):
    """The heads of every sequence, one element (not finite) or all of them
    (times a power of two)."""
    q = q.clone()
    for h in heads:
        if bad in (INF, -INF) or bad != bad:
            q[:, h, h % q.shape[2]] = bad
        else:
            q[:, h] *= bad
    return q


@pytest.mark.parametrize("dtype,bad", [(torch.bfloat16, INF), (torch.bfloat16, float("nan")), (torch.bfloat16, -INF), (torch.bfloat16, 2.0 ** 60),
                                       (torch.bfloat16, 2.0 ** 124), (torch.bfloat16, 2.0 ** -60), (torch.float16, INF), (torch.float16, float("nan")),
                                       (torch.float16, 2.0 ** 13), (torch.float16, 2.0 ** -14)])
@pytest.mark.parametrize("G,H,D,BS", [(4, 4, 128, 16), (8, 2, 64, 32), (16, 2, 128, 32), (9, 1, 64, 16), (2, 3, 128, 64)])
def test_one_head_apart(dtype, bad, G, H, D, BS):
    ctx = [1, 60, 300, 33]
    bt, P = R.tables(ctx, BS, seed=G)
    cache, vals, tops = U.make_cache(pkv, P, BS, H, D, seed=G)
    clean = rand((len(ctx), G * H, D), 3, dtype)
    apart = sorted({0, G - 1, G * H - 1 - G // 2} & set(range(G * H)))[:2 if G > 2 else 1]
    q = spoil(clean, apart, bad)
    cl = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    parts = U.decode_parts(clean, vals, tops, bt, ctx, D ** -0.5)
    rest = [h for h in range(G * H) if h not in apart]
    pick = lambda t: t[:, rest] if t.dim() > 1 else t  # noqa: E731
    for splits in (0, 1):
        out = pkv.paged_decode(q.to(DEV), cache, bt.to(DEV), cl, num_splits=splits)
        U.close(out[:, rest], tuple(pick(t) for t in parts), 4.5, dtype, D)
    if 0 < bad < 1:                               # the small ones are right as well
        parts = U.decode_parts(q, vals, tops, bt, ctx, D ** -0.5)
        U.close(pkv.paged_decode(q.to(DEV), cache, bt.to(DEV), cl), parts, 4.5, dtype, D)


@pytest.mark.parametrize("G", [3, 12])
@pytest.mark.parametrize("big", [2.0 ** 124, 2.0 ** 118, 2.0 ** -100])
def test_heads_of_the_types_largest(big, G):
    """Scores of ordinary size from queries at both ends of bf16's range."""
    ctx = [90, 20]
    bt, P = R.tables(ctx, 32)
    cache, vals, tops = U.make_cache(pkv, P, 32, 2, 64)
    q = rand((2, 2 * G, 64), 3, torch.bfloat16).clamp(-3.9, 3.9) * big
    sm = 0.125 / big
    if sm == 0 or sm > 1e38:
        sm = 1e37
    out = pkv.paged_decode(q.to(DEV), cache, bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV), sm_scale=sm)
    U.close(out, U.decode_parts(q, vals, tops, bt, ctx, sm), 4.5, torch.bfloat16, 64)


def test_one_hot_scores():
    """Scores near fp32's end pick one key."""
    ctx, D = [70], 64
    bt, P = R.tables(ctx, 32)
    cache, vals, _ = U.make_cache(pkv, P, 32, 1, D)
    q = torch.full((1, 2, D), 2.0 ** 100, dtype=torch.bfloat16)
    q[:, 1] = rand((1, D), 1, torch.bfloat16)
    out = pkv.paged_decode(q.to(DEV), cache, bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV))
    pos = torch.arange(ctx[0])
    at = bt[0].long()[pos // 32], pos % 32
    best = int((vals[0][at][:, 0].sum(-1)).argmax())
    assert float((out[0, 0].double().cpu() - vals[1][at][best, 0]).abs().max()) <= 2.0 ** -7 * 4.5
