"""paged_prefill over caches with scales per row or per block that lie far
apart, seen and unseen: a token's scale is no matter of a row that does not
see it, and a row's result is its own whatever the other scales are."""
import pytest
import torch

from tests import prompt_refs as R
from tests import scale_refs as S

pytestmark = pytest.mark.gpu

DEV = "cuda"
FORMS = [("e4m3", "token"), ("e4m3", "block"), ("e5m2", "token"), ("i8", "token"), ("i8", "block"), ("u3", "token")]


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_num_gb300 as P
    P.lib()
    return P


def attend(pkv, q, cache, bt, new, ctx):
    st = [0]
    for n in new:
        st.append(st[-1] + n)
    dev = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (st, ctx)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pkv.paged_prefill(q.to(DEV), cache, bt.to(DEV), *dev, err_flag=err)
    assert int(err.item()) == 0
    return st, out.cpu()


def compare(out, q, kv, vv, vs, bt, st, ctx, kind, dtype, rows=None):
    D = q.shape[2]
    ref = R.prefill(q, kv, vv, bt, st, ctx, D ** -0.5)
    big = S.lead(q, kv, vs, bt, st, ctx, D ** -0.5)
    rows = torch.arange(q.shape[0]) if rows is None else rows
    assert torch.isfinite(out[rows]).all()
    ref, big = tuple(x[rows] for x in ref), big[rows]
    d = (out[rows].double() - ref[0]).abs()
    tol = S.tolerance(ref, big, kind, dtype, D)
    assert torch.isfinite(tol).all()
    assert (d <= tol).all(), "worst %g of its tolerance" % float((d / tol).max())


def queries(T, H, D, dtype, seed, amp=1.0):
    return (torch.randn((T, H, D), generator=torch.Generator().manual_seed(seed)) * amp).to(dtype)


def shape_scales(bt, P, BS, H, kind, scales, at, factor):
    """Flat V scales but for token `at` of sequence 0 (per block: its block)."""
    vs = S.flat_scale(kind, (P, BS, H), amp=2.0 ** -12 if kind == "u3" else 1.0)
    blk = int(bt[0, at // BS])
    if scales == "block":
        vs[blk] *= factor
    else:
        vs[blk, at % BS] *= factor
    return vs


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [3, 8, 14, 22, 26, 60])
@pytest.mark.parametrize("kind,scales", FORMS)
def test_one_large_scale(pkv, kind, scales, bits, dtype):
    """One token (block) whose V scale is 2^bits times the others': rows before
    it are as if it had the others' scale, bit for bit; rows that see it are right."""
    if kind == "u3" and bits > 22:
        pytest.skip("f16 scales do not lie so far apart")
    if dtype == torch.float16 and bits > 14:
        pytest.skip("outputs beyond f16")
    H, G, D, BS, n, at = 2, 4, 128, 16, 300, 176
    bt, P = R.tables([n], BS, seed=bits)
    q = queries(n, H * G, D, dtype, 1)
    ks = S.flat_scale(kind, (P, BS, H), 0.5)
    outs = []
    for f in (1.0, 2.0 ** bits):
        vs = shape_scales(bt, P, BS, H, kind, scales, at, f)
        cache, kv, vv = S.coded_cache(pkv, kind, scales, ks, vs, D, seed=3)
        st, out = attend(pkv, q, cache, bt, [n], [n])
        compare(out, q, kv, vv, vs, bt, st, [n], kind, dtype)
        outs.append(out)
    assert torch.equal(outs[0][:at], outs[1][:at])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), 1e38])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("kind,scales", FORMS)
def test_hidden_scale_of_no_use(pkv, kind, scales, what, value, D):
    """A later token's scale that is infinite, NaN or next to the largest
    number: the rows before it are right."""
    H, G, BS, n, at = 2, 4, 16, 200, 144
    bt, P = R.tables([n], BS, seed=7)
    q = queries(n, H * G, D, torch.bfloat16, 2)
    ks, vs = S.flat_scale(kind, (P, BS, H), 0.5), S.flat_scale(kind, (P, BS, H))
    cache, kv, vv = S.coded_cache(pkv, kind, scales, ks, vs, D, seed=5)
    blk = int(bt[0, at // BS])
    if kind == "u3":
        (cache.k_qscale if what == "k" else cache.v_qscale)[blk, 0] = min(value, 65504.0)
    elif scales == "block":
        (cache.k_scales if what == "k" else cache.v_scales)[blk] = value
    else:
        (cache.k_scales if what == "k" else cache.v_scales)[blk, 0] = value
    st, out = attend(pkv, q, cache, bt, [n], [n])
    compare(out, q, kv, vv, vs, bt, st, [n], kind, torch.bfloat16, torch.arange(at))
    if value != value:                       # rows that see a NaN are NaN
        assert torch.isnan(out[at:]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind,scales", FORMS)
def test_scales_spread_over_many_powers_of_two(pkv, kind, scales, dtype):
    """Every row's V scale drawn over 2^-20 .. 2^4 (f16 ones 2^-14 .. 2^4), in
    prompts, chunks and few rows over a long context (split and joined)."""
    H, G, D, BS = 2, 4, 128, 16
    new, ctx = [150, 3, 40, 1], [150, 900, 400, 3000]
    bt, P = R.tables(ctx, BS, seed=9)
    g = torch.Generator().manual_seed(10)
    e = torch.randint(-14 if kind == "u3" else -20, 5, (P, 1 if scales == "block" else BS, H), generator=g)
    vs = S.flat_scale(kind, (P, BS, H)) * torch.exp2(e.float())
    if kind == "u3":
        vs = vs.clamp(min=2.0 ** -14)
    ks = S.flat_scale(kind, (P, BS, H), 0.5)
    cache, kv, vv = S.coded_cache(pkv, kind, scales, ks, vs, D, seed=11)
    q = queries(sum(new), H * G, D, dtype, 12)
    st, out = attend(pkv, q, cache, bt, new, ctx)
    compare(out, q, kv, vv, vs, bt, st, ctx, kind, dtype)


@pytest.mark.parametrize("kind,scales", FORMS)
def test_heavy_small_and_light_large(pkv, kind, scales):
    """One token has nearly all the weight and a small V scale, the others next
    to no weight and a scale up to 2^40 (f16: 2^13) times as large."""
    H, G, D, BS, c = 1, 8, 128, 16, 700
    n = 30
    bt, P = R.tables([c], BS, seed=13)
    for bits, strength in ((13, 4.0), (40, 12.0)):
        if kind == "u3" and bits > 13:
            continue
        ks, vs = S.flat_scale(kind, (P, BS, H), 0.05), S.flat_scale(kind, (P, BS, H), 1.0 if kind == "u3" else 2.0 ** (bits - 20))
        at = 333
        blk = int(bt[0, at // BS])
        if scales == "block":
            vs[blk] *= 2.0 ** -bits
        else:
            vs[blk, at % BS] *= 2.0 ** -bits
        cache, kv, vv = S.coded_cache(pkv, kind, scales, ks, vs, D, seed=14)
        # queries along that token's key
        k = kv[blk, at % BS, 0]
        q = (k / k.norm() ** 2 * D ** 0.5 * strength * 2.0).expand(n, H * G, D).to(torch.bfloat16)
        st, out = attend(pkv, q, cache, bt, [n], [c])
        compare(out, q, kv, vv, vs, bt, st, [c], kind, torch.bfloat16)


@pytest.mark.parametrize("kind,scales", [("e4m3", "token"), ("e4m3", "block"), ("i8", "token"), ("e5m2", "block")])
@pytest.mark.parametrize("bits", [-60, -30, 30, 60])
def test_all_scales_small_or_large(pkv, kind, scales, bits):
    """K and V scales whose common power of two is far from one."""
    H, G, D, BS = 2, 4, 64, 16
    new, ctx = [70, 2], [200, 1500]
    bt, P = R.tables(ctx, BS, seed=15)
    ks, vs = S.flat_scale(kind, (P, BS, H), 2.0 ** (bits / 2)), S.flat_scale(kind, (P, BS, H), 2.0 ** bits)
    cache, kv, vv = S.coded_cache(pkv, kind, scales, ks, vs, D, seed=16)
    q = queries(sum(new), H * G, D, torch.bfloat16, 17, 2.0 ** (-bits / 2))
    st, out = attend(pkv, q, cache, bt, new, ctx)
    compare(out, q, kv, vv, vs, bt, st, ctx, kind, torch.bfloat16)


@pytest.mark.parametrize("kind", ["e4m3", "u3"])
def test_scales_of_zero(pkv, kind):
    """Rows whose K or V scale is zero have the value zero."""
    H, G, D, BS = 2, 4, 128, 16
    new, ctx = [150, 2], [150, 1500]
    bt, P = R.tables(ctx, BS, seed=18)
    g = torch.Generator().manual_seed(19)
    ks, vs = S.flat_scale(kind, (P, BS, H), 0.5), S.flat_scale(kind, (P, BS, H))
    ks[torch.rand((P, BS, H), generator=g) < 0.2] = 0.0
    vs[torch.rand((P, BS, H), generator=g) < 0.2] = 0.0
    cache, kv, vv = S.coded_cache(pkv, kind, "token", ks, vs, D, seed=20)
    q = queries(sum(new), H * G, D, torch.bfloat16, 21)
    st, out = attend(pkv, q, cache, bt, new, ctx)
    compare(out, q, kv, vv, vs, bt, st, ctx, kind, torch.bfloat16)


def test_padded_pool_scales(pkv):
    """Scales behind the contexts and of blocks that no table names hold NaN."""
    H, G, D, BS = 2, 4, 128, 16
    new, ctx = [41, 3], [41, 333]
    for kind, scales in FORMS:
        bt, P = R.tables(ctx, BS, seed=22)
        ks, vs = S.flat_scale(kind, (P, BS, H), 0.5), S.flat_scale(kind, (P, BS, H))
        cache, kv, vv = S.coded_cache(pkv, kind, scales, ks, vs, D, seed=23)
        seen = torch.zeros((P, BS), dtype=torch.bool)
        for b, c in enumerate(ctx):
            for t in range(c):
                seen[bt[b, t // BS], t % BS] = True
        pair = (cache.k_qscale, cache.v_qscale) if kind == "u3" else (cache.k_scales, cache.v_scales)
        for t in pair:
            t[(~seen.any(1) if scales == "block" else ~seen).to(DEV)] = float("nan")
        q = queries(sum(new), H * G, D, torch.bfloat16, 24)
        st, out = attend(pkv, q, cache, bt, new, ctx)
        compare(out, q, kv, vv, vs, bt, st, ctx, kind, torch.bfloat16)


@pytest.mark.parametrize("first", ["heavy", "large"])
@pytest.mark.parametrize("n,c", [(1, 300), (40, 300), (300, 700), (2, 9000)])
def test_weights_and_scales_at_opposite_ends(pkv, n, c, first):
    """Half of the context has nearly all the weight and V scales of 2^-70, the
    other half next to none and scales of 2^70: the sum of weights is the
    first half's, though its products are nothing beside the other's."""
    H, G, D, BS = 1, 4, 128, 16
    bt, P = R.tables([c], BS, seed=25)
    heavy = torch.arange(c) < c // 2 if first == "heavy" else torch.arange(c) >= c // 2
    blk, off = bt[0].long()[torch.arange(c) // BS], torch.arange(c) % BS
    ks, vs = torch.full((P, BS, H), 2.0 ** -20), torch.full((P, BS, H), 2.0 ** 70)
    ks[blk[heavy], off[heavy]] = 2.0 ** -4
    vs[blk[heavy], off[heavy]] = 2.0 ** -70
    cache, kv, vv = S.coded_cache(pkv, "e4m3", "token", ks, vs, D, seed=26)
    # the heavy keys' codes: 4 everywhere, against positive queries
    code = torch.full((), 4.0).to(torch.float8_e4m3fn).view(torch.uint8)
    cache.k_cache.view(torch.uint8)[blk[heavy].to(DEV), off[heavy].to(DEV)] = int(code)
    kv[blk[heavy], off[heavy]] = 4.0 * 2.0 ** -4
    q = queries(n, H * G, D, torch.bfloat16, 27).abs() * 2
    st, out = attend(pkv, q, cache, bt, [n], [c])
    compare(out, q, kv, vv, vs, bt, st, [c], "e4m3", torch.bfloat16)


@pytest.mark.parametrize("kind,scales", [("e4m3", "token"), ("i8", "block"), ("e4m3", "head"), ("bf16", "head")])
@pytest.mark.parametrize("bits", [-85, 85])
def test_queries_and_keys_at_opposite_ends(pkv, kind, scales, bits):
    """Queries of 2^-bits and keys of 2^bits: ordinary scores."""
    H, G, D, BS = 2, 4, 128, 16
    new, ctx = [130, 2], [130, 900]
    bt, P = R.tables(ctx, BS, seed=28)
    if scales == "head":
        cache, kv, vv = R.make_cache(pkv, kind, P, BS, H, D, seed=29)
        vs = torch.ones((P, BS, H)) if kind == "bf16" else cache.v_scale.cpu().expand(P, BS, H)
        if kind == "bf16":
            cache.k_cache *= 2.0 ** bits
        else:
            cache.k_scale *= 2.0 ** bits
        kv = kv * 2.0 ** bits
    else:
        ks, vs = S.flat_scale(kind, (P, BS, H), 2.0 ** bits), S.flat_scale(kind, (P, BS, H))
        cache, kv, vv = S.coded_cache(pkv, kind, scales, ks, vs, D, seed=30)
    q = queries(sum(new), H * G, D, torch.bfloat16, 31, 2.0 ** -bits)
    st, out = attend(pkv, q, cache, bt, new, ctx)
    S.CMAX.setdefault("bf16", 8.0)
    compare(out, q, kv, vv, vs, bt, st, ctx, kind, torch.bfloat16)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [1e-34, -1e-34, 0.0])
def test_a_tiny_softmax_scale(pkv, kind, scale):
    """Queries and keys of 1e17, a scale of 1e-34: scores of a few units; and a
    scale of zero, under which all weights are alike."""
    H, G, D, BS, new, ctx = 2, 4, 128, 16, [130, 2], [130, 900]
    bt, P = R.tables(ctx, BS, seed=32)
    cache, kv, vv = R.make_cache(pkv, kind, P, BS, H, D, seed=33)
    if kind == "bf16":
        cache.k_cache *= 2.0 ** 56
    else:
        cache.k_scale *= 2.0 ** 56
    kv = kv * 2.0 ** 56
    q = queries(sum(new), H * G, D, torch.bfloat16, 34, 2.0 ** 54)
    st = [0, 130, 132]
    dev = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (st, ctx)]
    out = pkv.paged_prefill(q.to(DEV), cache, bt.to(DEV), *dev, sm_scale=scale).cpu()
    ref = R.prefill(q, kv, vv, bt, st, ctx, float(torch.tensor(scale)))
    assert ((out.double() - ref[0]).abs() <= R.prefill_tolerance(*ref, 0.0, torch.bfloat16, D)).all()
