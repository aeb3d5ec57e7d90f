"""paged_decode over caches with scales per row or per block of any size,
among them those that kv_append_dynamic stores, against attention in float64."""
import pytest
import torch

from tests import prompt_refs as R
from tests import scale_refs as S

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_num_gb300 as P
    P.lib()
    return P


def compare(pkv, q, cache, kv, vv, vs, bt, ctx, kind, splits=0, ks=0.0):
    D = q.shape[2]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pkv.paged_decode(q.to(DEV), cache, bt.clamp(min=0).to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV),
                           num_splits=splits, err_flag=err).cpu()
    assert int(err.item()) == 0
    st = list(range(len(ctx) + 1))
    ref = R.prefill(q, kv, vv, bt, st, ctx, D ** -0.5)
    tol = S.tolerance(ref, S.lead(q, kv, vs, bt, st, ctx, D ** -0.5), kind, q.dtype, D)
    # int8 codes are code + 1152 in the products, whose sums the offsets' sums are taken from: each step of
    # 16 adds up numbers of up to 1279 and is off by at most 2^-23 of the sum, and so is the offset's
    if kind == "i8":
        score = 2 * (D / 16 + 2) * 2.0 ** -23 * 1279 * q.double().abs().sum(-1) * ks * D ** -0.5
        total = S.lead(q, kv, vs, bt, st, ctx, D ** -0.5, total=True)
        tol = tol + (2 * score[..., None]) * ref[1] + \
            (2 * (ref[3][:, None] / 16 + 8) * 2.0 ** -23 * 1279 * total)[..., None]
    d = (out.double() - ref[0]).abs()
    assert torch.isfinite(out).all() and (d <= tol).all(), "worst %g of its tolerance" % float((d / tol).max())


@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("amp", [1e-4, 3.0, 1e4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_decode_of_a_dynamic_append(pkv, kind, dtype, amp, D, splits):
    """V rows of any amplitude, appended with computed scales and decoded."""
    if dtype == torch.float16 and amp == 1e4:
        amp = 1e3
    H, G, BS, ctx = 4, 4, 16, [1, 37, 300, 1500]
    bt, P = R.tables(ctx, BS, seed=1)
    g = torch.Generator().manual_seed(2)
    slots = torch.cat([bt[b].long()[torch.arange(c) // BS] * BS + torch.arange(c) % BS for b, c in enumerate(ctx)])
    k = torch.randn((sum(ctx), H, D), generator=g).to(dtype)
    v = (torch.randn((sum(ctx), H, D), generator=g) * amp).to(dtype)
    cache = pkv.KVCache.allocate(kind, P, BS, H, D, fill=0, scale_mode="token")
    pkv.kv_append_dynamic(k.to(DEV), v.to(DEV), slots.to(DEV), cache)
    vals = []
    for buf, sc in ((cache.k_cache, cache.k_scales), (cache.v_cache, cache.v_scales)):
        vals.append(buf.cpu().view(R.CODE[kind]).double() * sc.cpu().double()[..., None])
    q = torch.randn((len(ctx), H * G, D), generator=g).to(dtype)
    compare(pkv, q, cache, *vals, cache.v_scales.cpu().double(), bt, ctx, kind, splits)


@pytest.mark.parametrize("G", [4, 12])
@pytest.mark.parametrize("kind,scales", [("e4m3", "token"), ("e4m3", "block"), ("e5m2", "token"), ("i8", "token"), ("i8", "block")])
def test_scales_spread_over_many_powers_of_two(pkv, kind, scales, G):
    H, D, BS, ctx = 4, 128, 16, [5, 300, 2000]
    bt, P = R.tables(ctx, BS, seed=3)
    g = torch.Generator().manual_seed(4)
    e = torch.randint(-30, 5, (P, 1 if scales == "block" else BS, H), generator=g)
    vs = S.flat_scale(kind, (P, BS, H)) * torch.exp2(e.float())
    ks = S.flat_scale(kind, (P, BS, H), 0.5)
    cache, kv, vv = S.coded_cache(pkv, kind, scales, ks, vs, D, seed=5)
    q = torch.randn((len(ctx), H * G, D), generator=g).bfloat16()
    compare(pkv, q, cache, kv, vv, vs, bt, ctx, kind, ks=float(ks.max()))


@pytest.mark.parametrize("bits", [-40, 40])
@pytest.mark.parametrize("kind,scales", [("e4m3", "token"), ("i8", "block")])
def test_all_scales_small_or_large(pkv, kind, scales, bits):
    H, G, D, BS, ctx = 4, 4, 128, 16, [5, 300, 2000]
    bt, P = R.tables(ctx, BS, seed=6)
    vs = S.flat_scale(kind, (P, BS, H)) * 2.0 ** bits
    ks = S.flat_scale(kind, (P, BS, H), 0.5)
    cache, kv, vv = S.coded_cache(pkv, kind, scales, ks, vs, D, seed=7)
    q = torch.randn((len(ctx), H * G, D), generator=torch.Generator().manual_seed(8)).bfloat16()
    compare(pkv, q, cache, kv, vv, vs, bt, ctx, kind, ks=float(ks.max()))


@pytest.mark.parametrize("first", ["heavy", "large"])
@pytest.mark.parametrize("c", [100, 3000])
def test_weights_and_scales_at_opposite_ends(pkv, c, first):
    """Half of the context has nearly all the weight and V scales of 2^-38, the
    other half next to none and scales of 2^38."""
    H, G, D, BS = 4, 4, 128, 16
    bt, P = R.tables([c], BS, seed=9)
    heavy = torch.arange(c) < c // 2 if first == "heavy" else torch.arange(c) >= c // 2
    blk, off = bt[0].long()[torch.arange(c) // BS], torch.arange(c) % BS
    ks, vs = torch.full((P, BS, H), 2.0 ** -20), torch.full((P, BS, H), 2.0 ** 38)
    ks[blk[heavy], off[heavy]] = 2.0 ** -4
    vs[blk[heavy], off[heavy]] = 2.0 ** -38
    cache, kv, vv = S.coded_cache(pkv, "e4m3", "token", ks, vs, D, seed=10)
    code = torch.full((), 4.0).to(torch.float8_e4m3fn).view(torch.uint8)
    cache.k_cache.view(torch.uint8)[blk[heavy].to(DEV), off[heavy].to(DEV)] = int(code)
    kv[blk[heavy], off[heavy]] = 4.0 * 2.0 ** -4
    q = (torch.randn((1, H * G, D), generator=torch.Generator().manual_seed(11)).abs() * 2).bfloat16()
    compare(pkv, q, cache, kv, vv, vs, bt, [c], "e4m3")
