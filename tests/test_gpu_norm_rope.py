"""Norm and rotation of query and key heads against the formula in 64 bits, and
the fused append against the separate calls, byte for byte."""
import math

import pytest
import torch

import paged_kv_cache_num_gb300 as pkv
from paged_kv_cache_num_gb300 import pkv as P_

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


def rand(shape, seed, dtype=torch.float32, amp=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * amp).to(dtype)


def table(rot, n=5000):
    half = rot // 2
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    return torch.cat([a.cos(), a.sin()], -1).float()


def turned(x, w, cs, pos, eps, pairs):
    """The formula in float64, and the sum of the two products' magnitudes."""
    x = x.double()
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    rot = cs.shape[1]
    half = rot // 2
    c, s = cs[pos.long()].double()[:, None].split(half, -1)
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
    y, big = x.clone(), x.abs()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    big[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
    big[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, big


def check(got, want, big, dtype, D):
    """One rounding to the type, and in fp32 before it, in roundings of 2^-24 of the
    products' magnitudes: the mean's at most D / 8 + 5 sums, halved by the root; the
    root to two steps of 2^-23, that is 4; weight times cosine, two products, their sum
    and the product with the root, 4: D / 16 + 11 (values below the normal range: half of
    the least step)."""
    h = torch.finfo(dtype).eps / 2
    tol = h * want.abs() * (1 + h) + (D / 16 + 11) * 2.0 ** -24 * big * (1 + 2 * h) + torch.finfo(dtype).smallest_normal * h
    err = (got.double().cpu() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", [(1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (7, 5, 3, 64, 16), (65, 9, 1, 128, 32), (300, 4, 4, 128, 96),
                                            (3, 0, 2, 64, 32), (2, 3, 0, 64, 48), (2500, 16, 2, 128, 64), (1111, 40, 10, 64, 64), (5003, 9, 5, 128, 64)])
def test_norm_rope(dtype, pairs, T, Hq, Hkv, D, rot):
    q, k = rand((T, Hq, D), 1, dtype), rand((T, Hkv, D), 2, dtype, 30.0)
    wq, wk = 1 + rand((D,), 3, amp=0.3), 1 + rand((D,), 4, amp=0.3)
    cs = table(rot)
    pos = torch.randint(0, cs.shape[0], (T,), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    for weights in ((wq, wk), (wq.to(dtype), wk.to(dtype)), (None, None), (wq, None), (None, wk.to(dtype))):
        qo, ko = pkv.norm_rope(q.to(DEV), k.to(DEV), cs.to(DEV), pos.to(DEV), *(None if w is None else w.to(DEV) for w in weights), eps=EPS, interleaved=pairs)
        for got, x, w in ((qo, q, weights[0]), (ko, k, weights[1])):
            check(got, *turned(x, w, cs, pos, EPS, pairs), dtype, D)


def test_no_tokens():
    z = torch.zeros((0, 4, 64), dtype=torch.float16, device=DEV)
    q, k = pkv.norm_rope(z, z, table(64).to(DEV), torch.zeros(0, dtype=torch.int32, device=DEV))
    assert q.shape == k.shape == z.shape


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_rows_at_the_edges(dtype):
    """Zeros, single elements, large and small rows; eps of zero and of one."""
    D = 128
    rows = torch.zeros((8, 1, D))
    rows[1, 0, 5], rows[2, 0, 127], rows[3] = 7, -3e-3, rand((1, D), 1) * 1000
    rows[4], rows[5], rows[6, 0, ::2], rows[7] = rand((1, D), 2) * 1e-4, 60000.0, 1.0, -2.0
    x = rows.to(dtype)
    w = rand((D,), 3)
    cs, pos = table(D), torch.arange(8, dtype=torch.int32) * 600
    for eps in (1.0, 1e-5):
        q, k = pkv.norm_rope(x.to(DEV), x.to(DEV), cs.to(DEV), pos.to(DEV), w.to(DEV), w.to(DEV), eps=eps)
        check(q, *turned(x, w, cs, pos, eps, False), dtype, D)
        assert torch.equal(q, k)
    # a row that is not finite is no matter of the others
    x[3, 0, 9] = float("nan")
    x[5, 0, 0] = float("inf")
    q = pkv.norm_rope(x.to(DEV), x.to(DEV), cs.to(DEV), pos.to(DEV), w.to(DEV), w.to(DEV))[0]
    ok = torch.tensor([0, 1, 2, 4, 6, 7])
    want, big = turned(x, w, cs, pos, 1e-6, False)
    check(q.cpu()[ok], want[ok], big[ok], dtype, D)
    assert q[3].isnan().all()


def test_without_norm_and_rotation_the_bits_stay():
    """Elements behind the rotation of rows without a norm are copied, NaN and all."""
    x = torch.randint(-2 ** 15, 2 ** 15, (50, 3, 128), generator=torch.Generator().manual_seed(1)).to(torch.int16).view(torch.float16)
    q, _ = pkv.norm_rope(x.to(DEV), x.to(DEV), table(32).to(DEV), torch.zeros(50, dtype=torch.int32, device=DEV))
    same = q.cpu()[..., 32:].view(torch.int16) == x[..., 32:].view(torch.int16)
    assert (same | x[..., 32:].isnan()).all() and (q.cpu().isnan() == x.isnan())[..., 32:].all()


@pytest.mark.parametrize("pairs", [False, True])
def test_in_place_strided_and_unaligned(pairs):
    """Views of the fused projection, onto themselves and into wider buffers."""
    T, Hq, Hkv, D = 33, 6, 2, 64
    for dtype in (torch.float16, torch.bfloat16):
        for shift in (0, 1, 4):
            fused = rand((T, Hq + 2 * Hkv, D + 8), 1, dtype)
            w, cs = rand((D,), 2), table(32)
            pos = torch.arange(T * 2, dtype=torch.int32)[::2]
            part = lambda f: (f[:, :Hq, shift:shift + D], f[:, Hq:Hq + Hkv, shift:shift + D])  # noqa: E731
            q, k = part(fused)
            want = [turned(x, w, cs, pos, EPS, pairs) for x in (q, k)]
            dev = fused.to(DEV)
            qd, kd = part(dev)
            pd = torch.arange(T * 2, dtype=torch.int32, device=DEV)[::2]
            qo, ko = pkv.norm_rope(qd, kd, cs.to(DEV), pd, w.to(DEV), w.to(DEV), eps=EPS, interleaved=pairs)
            pkv.norm_rope(qd, kd, cs.to(DEV), pd, w.to(DEV), w.to(DEV), eps=EPS, interleaved=pairs, q_out=qd, k_out=kd)
            for a, b, x in zip((qo, ko), (qd, kd), want):
                check(a, *x, dtype, D)
                assert torch.equal(a, b)
            rest = torch.ones(fused.shape, dtype=torch.bool)
            for x in part(rest):
                x.zero_()
            assert torch.equal(dev.cpu()[rest], fused[rest])          # values and borders as they were


@pytest.mark.parametrize("many", [1, 600])
def test_padding_and_bad_positions(many):
    """Few tokens, a part of one to a warp, and many, whole ones."""
    T, D = 9 * many, 64
    x = rand((T, 2, D), 1, torch.float16)
    cs = table(64, 50)
    pos = torch.tensor([0, -1, 49, 50, 7, -2 ** 31, 2 ** 31 - 1, 3, -1], dtype=torch.int32).repeat(many)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((T, 2, D), 5.0, dtype=torch.float16, device=DEV)
    q, k = pkv.norm_rope(x.to(DEV), x.to(DEV), cs.to(DEV), pos.to(DEV), q_out=out, err_flag=err)
    assert err.item() == P_.DEVERR_POS_RANGE
    ok = (pos >= 0) & (pos < 50)
    want, big = turned(x[ok], None, cs, pos[ok], EPS, False)
    check(q.cpu()[ok], want, big, torch.float16, D)
    assert (q.cpu()[~ok] == 5).all() and (k.cpu()[~ok] == 0).all()
    err.zero_()
    cache = pkv.KVCache.allocate("f16", 2, 16, 2, D, fill=0)
    slots = torch.tensor([3, 4, -1, 5, 32, 6, 7, 8, 9] + [-1, -7, 1 << 40] * 3 * (many - 1))
    q2 = pkv.norm_rope_append(x.to(DEV), x.to(DEV), x.to(DEV), cs.to(DEV), pos.to(DEV), slots.to(DEV), cache, err_flag=err)
    assert err.item() == P_.DEVERR_POS_RANGE | P_.DEVERR_SLOT_RANGE
    assert torch.equal(q2[ok.to(DEV)], q[ok.to(DEV)])              # queries whether or not the row is stored
    stored = [t for t in range(T) if ok[t] and 0 <= slots[t] < 32]
    rows = cache.v_cache.view(32, 2, D).cpu()
    assert torch.equal(rows[slots[stored]], x[stored])
    rest = [s for s in range(32) if s not in slots[stored].tolist()]
    assert (rows[rest] == 0).all() and (cache.k_cache.view(32, 2, D).cpu()[rest] == 0).all()


def make(kind, P, BS, H, D, mode="head", layout="flash"):
    kw = {}
    if kind in ("e4m3", "e5m2", "i8"):
        g = torch.Generator().manual_seed(9)
        if mode == "head":
            kw = {"k_scale": (torch.rand(H, generator=g) * 0.02 + 0.005).to(DEV), "v_scale": (torch.rand(H, generator=g) * 0.02 + 0.005).to(DEV)}
        elif mode == "block":
            kw = {n: (torch.rand((P, H), generator=g) * 0.02 + 0.005).to(DEV) for n in ("k_scales", "v_scales")}
        kw["scale_mode"] = mode
    return pkv.KVCache.allocate(kind, P, BS, H, D, fill=0x11, layout=layout, **kw)


CACHES = [("same", "head", "flash"), ("same", "head", "xvec"), ("e4m3", "head", "flash"), ("e4m3", "block", "xvec"), ("e4m3", "token", "flash"),
          ("e5m2", "token", "xvec"), ("i8", "block", "flash"), ("i8", "token", "flash"), ("u4", "head", "flash"), ("u3", "head", "flash")]


@pytest.mark.parametrize("kind,mode,layout", CACHES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,Hq,H,D,BS", [(1, 4, 1, 64, 16), (70, 7, 3, 128, 16), (2100, 8, 8, 128, 32), (900, 6, 5, 64, 24), (5003, 6, 3, 64, 16)])
def test_append_equals_the_separate_calls(kind, mode, layout, dtype, T, Hq, H, D, BS):
    kind = {torch.float16: "f16", torch.bfloat16: "bf16"}[dtype] if kind == "same" else kind
    P = T // BS + 2
    fused = rand((T, Hq + 2 * H, D), 1, dtype, 2.0).to(DEV)
    fused[0, Hq + H] = 0                                             # a value row of zeros
    q, k, v = fused.split([Hq, H, H], 1)
    wq, wk = (1 + rand((D,), 3, dtype, 0.3)).to(DEV), (1 + rand((D,), 4, dtype, 0.3)).to(DEV)
    cs = table(D // 2).to(DEV)
    g = torch.Generator().manual_seed(T)
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32).to(DEV)
    slots = torch.randperm(P * BS, generator=g)[:T].to(DEV)
    if T > 3:
        slots[1] = -1
    one, two = make(kind, P, BS, H, D, mode, layout), make(kind, P, BS, H, D, mode, layout)
    for pairs in (False, True):
        qf = pkv.norm_rope_append(q, k, v, cs, pos, slots, one, wq, wk, interleaved=pairs)
        qs, ks = pkv.norm_rope(q, k, cs, pos, wq, wk, interleaved=pairs)
        (pkv.kv_append_dynamic if mode == "token" else pkv.kv_append)(ks, v.contiguous(), slots, two)
        assert torch.equal(qf, qs)
        for a, b in zip(one.tensors(), two.tensors()):
            assert torch.equal(a if a.dtype != torch.float32 else a.contiguous().view(torch.int32), b if b.dtype != torch.float32 else b.contiguous().view(torch.int32))


def test_dynamic_scales_of_rows_that_are_not_finite():
    """As kv_append_dynamic: the scale from the finite elements."""
    T, H, D = 6, 2, 64
    x = rand((T, H, D), 1, torch.bfloat16)
    x[1, 0, 3], x[2, 1, 5], x[3], x[4] = float("inf"), float("nan"), float("nan"), 0
    cs, pos, slots = table(64).to(DEV), torch.zeros(T, dtype=torch.int32, device=DEV), torch.arange(T, device=DEV)
    for kind in ("e4m3", "e5m2", "i8"):
        one, two = make(kind, 1, 16, H, D, "token"), make(kind, 1, 16, H, D, "token")
        pkv.norm_rope_append(x.to(DEV), x.to(DEV), x.to(DEV), cs, pos, slots, one)
        pkv.kv_append_dynamic(pkv.norm_rope(x.to(DEV), x.to(DEV), cs, pos)[1], x.to(DEV), slots, two)
        for a, b in zip(one.tensors(), two.tensors()):
            assert torch.equal(a.contiguous().view(torch.uint8) if a.dtype != torch.float32 else a, b.contiguous().view(torch.uint8) if b.dtype != torch.float32 else b)


def test_captured_on_another_stream():
    T, Hq, H, D = 20, 4, 2, 128
    q, k, v = (rand((T, h, D), i, torch.bfloat16).to(DEV) for i, h in enumerate((Hq, H, H)))
    cs, pos, slots = table(D).to(DEV), torch.arange(T, dtype=torch.int32, device=DEV), torch.arange(T, device=DEV)
    cache = pkv.KVCache.allocate("u4", 2, 16, H, D, fill=0)
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pkv.norm_rope_append(q, k, v, cs, pos, slots, cache, q_out=out, stream=s)
    s.synchronize()
    want, first = out.clone(), [t.clone() for t in cache.tensors()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.norm_rope_append(q, k, v, cs, pos, slots, cache, q_out=out)
    out.zero_()
    for t in cache.tensors():
        t.zero_()
    g.replay()
    assert torch.equal(out, want)
    for a, b in zip(cache.tensors(), first):
        assert torch.equal(a, b)


def test_rotation_leaves_scores_that_depend_on_distance():
    """q at position a and k at b have the product of q at a + d and k at b + d."""
    D = 128
    q, k = rand((1, 1, D), 1, torch.float16), rand((1, 1, D), 2, torch.float16)
    cs = table(D).to(DEV)
    rot = lambda x, p: pkv.norm_rope(x.to(DEV), x.to(DEV), cs, torch.tensor([p], dtype=torch.int32, device=DEV))[0].double().cpu()  # noqa: E731
    near = float((rot(q, 17) * rot(k, 5)).sum())
    far = float((rot(q, 4017) * rot(k, 4005)).sum())
    # each product's two factors are rounded to f16, and the angles to fp32
    bound = 4 * (2.0 ** -11 + 2.0 ** -23) * float(q.double().norm() * k.double().norm())
    assert math.isfinite(near) and abs(near - far) <= bound
