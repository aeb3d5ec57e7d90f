"""The 4-bit cache on the GPU: appended codes bit for bit, rows read back,
decode and prefill against 64-bit attention over the dequantised cache."""
import itertools

import pytest
import torch

import paged_kv_cache_num_gb300 as pkv
from paged_kv_cache_num_gb300 import pkv as P_
from tests import prompt_refs as R
from tests import u4_refs as U

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rand(shape, seed, dtype, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * amp).to(dtype)


# ---------------------------------------------------------------- append and gather
def read(cache, slots):
    """(codes, scale, zero) of K and of V at slots, on the CPU."""
    BS = cache.block_size
    out = []
    for data, s, z in ((cache.k_cache, cache.k_qscale, cache.k_qzero), (cache.v_cache, cache.v_qscale, cache.v_qzero)):
        at = (slots // BS, slots % BS)
        out.append((U.numpy_codes(data.cpu()[at]), s.cpu()[at], z.cpu()[at]))
    return out


def check_append(k, v, slots, cache):
    """Appended rows and nothing else, in the whole pool."""
    for t in cache.tensors():
        t.fill_(0xA5)
    want = pkv.KVCache("u4", *(t.clone() for t in (cache.k_cache, cache.v_cache)), **{
        n: getattr(cache, n).clone() for n in ("k_qscale", "v_qscale", "k_qzero", "v_qzero")})
    pkv.kv_append(k.to(DEV), v.to(DEV), slots.to(DEV), cache)
    BS = cache.block_size
    ok = (slots >= 0) & (slots < cache.num_blocks * BS)
    blk, off = slots[ok].to(DEV) // BS, slots[ok].to(DEV) % BS
    for x, d, s, z in ((k, want.k_cache, want.k_qscale, want.k_qzero), (v, want.v_cache, want.v_qscale, want.v_qzero)):
        codes, scale, zero = U.quantise(x.cpu()[ok])
        d[blk, off], s[blk, off], z[blk, off] = U.pack4(codes).to(DEV), scale.to(DEV), zero.to(DEV)
    for n in ("k_cache", "v_cache", "k_qscale", "v_qscale", "k_qzero", "v_qzero"):
        a, b = getattr(cache, n), getattr(want, n)
        assert torch.equal(a, b), n


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,H,D,BS", [(1, 1, 64, 16), (1, 1, 128, 16), (5, 3, 128, 8), (33, 8, 128, 32), (700, 5, 64, 16), (3001, 8, 128, 16), (2500, 32, 64, 12)])
def test_append(dtype, T, H, D, BS):
    P = T // BS + 3
    slots = torch.randperm(P * BS, generator=torch.Generator().manual_seed(T))[:T]
    slots[T // 2] = -1 if T > 2 else slots[0]
    cache = pkv.KVCache.allocate("u4", P, BS, H, D)
    check_append(rand((T, H, D), 1, dtype), rand((T, H, D), 2, dtype, 3.0), slots, cache)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_append_of_rows_at_the_edges(dtype):
    """Zeros, equal numbers, one sign, the type's largest, subnormals, ties."""
    D = 128
    big = float(torch.finfo(dtype).max)
    tiny = float(torch.finfo(dtype).smallest_normal)
    g = torch.Generator().manual_seed(3)
    rows = [torch.zeros(D), torch.full((D,), 2.5), torch.full((D,), -0.75), torch.rand(D, generator=g) + 1, -torch.rand(D, generator=g) - 1,
            torch.full((D,), big), torch.randn(D, generator=g).sign() * big, torch.randn(D, generator=g) * tiny, torch.arange(D) * (tiny / 64),
            torch.arange(D) % 16 - 7.5, (torch.arange(D) % 31) * 0.5 - 7, torch.arange(D) * 0.25, -torch.arange(D) * 0.125, torch.zeros(D) - 0.0,
            torch.randn(D, generator=g) * 6e-8, torch.randn(D, generator=g) * 1e-3 + 100]
    x = torch.stack(rows).to(dtype)[:, None, :].repeat(1, 2, 1)
    x[:, 1] = -x[:, 1]
    T = x.shape[0]
    check_append(x, x.flip(0), torch.arange(T) * 2 + 1, pkv.KVCache.allocate("u4", 5, 16, 2, D))


def test_append_from_strided_and_unaligned_rows():
    T, H, D = 77, 3, 128
    for dtype in (torch.float16, torch.bfloat16):
        fused = rand((T, 2 * H + 1, D + 8), 5, dtype).to(DEV)
        slots = torch.randperm(96, generator=torch.Generator().manual_seed(5))[:T]
        for shift in (0, 1, 3):                   # off the 16-byte boundary
            k, v = fused[:, :H, shift:shift + D], fused[:, H:2 * H, shift:shift + D]
            check_append(k, v, slots, pkv.KVCache.allocate("u4", 6, 16, H, D))


def test_append_skips_and_flags():
    T, H, D = 6, 2, 64
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    cache = pkv.KVCache.allocate("u4", 2, 16, H, D, fill=7)
    slots = torch.tensor([-1, 32, -5, 1 << 40, 3, -1 << 60])
    k = rand((T, H, D), 1, torch.float16)
    k[0] = float("nan")
    pkv.kv_append(k.to(DEV), k.to(DEV), slots.to(DEV), cache, err_flag=err)
    assert err.item() == P_.DEVERR_SLOT_RANGE
    codes = read(cache, torch.arange(32))
    want = U.quantise(k[4])
    for c, s, z in codes:
        assert torch.equal(c[3], want[0]) and torch.equal(s[3], want[1]) and torch.equal(z[3], want[2])
        assert (z[torch.arange(32) != 3] == 7).all()


def test_append_of_no_tokens():
    cache = pkv.KVCache.allocate("u4", 2, 16, 2, 64)
    k = torch.zeros((0, 2, 64), dtype=torch.float16, device=DEV)
    pkv.kv_append(k, k, torch.zeros(0, dtype=torch.int64, device=DEV), cache)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,H,D,BS,hmaj", [(1, 1, 64, 16, True), (9, 2, 128, 8, False), (300, 5, 128, 32, True), (2000, 8, 64, 24, False), (4001, 8, 128, 16, True)])
def test_gather(dtype, T, H, D, BS, hmaj):
    P = T // BS + 2
    cache, vals, _ = U.make_cache(pkv, P, BS, H, D, seed=T, hmaj=hmaj)
    g = torch.Generator().manual_seed(T)
    slots = torch.randint(0, P * BS, (T,), generator=g)           # the same slot more than once
    k, v = pkv.kv_gather(cache, slots.to(DEV), dtype=dtype)
    for got, x in ((k, vals[0]), (v, vals[1])):
        # a code difference times an f16 scale is exact in float64: one rounding
        assert torch.equal(got.cpu(), x[slots // BS, slots % BS].to(dtype))


def test_gather_of_extreme_scales_and_zeros():
    """Zeros above 15 and scales from subnormal to infinite."""
    P, BS, H, D = 2, 16, 1, 64
    cache, _, _ = U.make_cache(pkv, P, BS, H, D)
    s = torch.tensor([0.0, 6e-8, 3e-5, 1.0, -2.0, 65504.0, float("inf"), float("nan")] * 4, dtype=torch.float16).view(P, BS, H)
    z = torch.tensor([0, 255, 16, 15] * 8, dtype=torch.uint8).view(P, BS, H)
    for n in ("k", "v"):
        getattr(cache, n + "_qscale").copy_(s)
        getattr(cache, n + "_qzero").copy_(z)
    slots = torch.arange(P * BS)
    codes = U.numpy_codes(cache.k_cache).view(P * BS, H, D)
    want = (codes.double() - z.view(-1, H, 1).double()) * s.view(-1, H, 1).double()
    for dtype in (torch.float16, torch.bfloat16):
        got = pkv.kv_gather(cache, slots.to(DEV), dtype=dtype)[0].cpu()
        assert torch.equal(torch.nan_to_num(got.float(), 7.0), torch.nan_to_num(want.to(dtype).float(), 7.0))
        assert torch.equal(got.isnan(), want.isnan())


def test_gather_keeps_rows_and_takes_strides():
    T, H, D = 40, 3, 128
    cache, vals, _ = U.make_cache(pkv, 4, 16, H, D)
    slots = torch.randint(0, 64, (T,), generator=torch.Generator().manual_seed(1))
    slots[::7] = -1
    for shift in (0, 1):
        out = torch.full((T, 2 * H, D + 8), 9.0, dtype=torch.float16, device=DEV)
        k, v = out[:, :H, shift:shift + D], out[:, H:, shift:shift + D]
        pkv.kv_gather(cache, slots.to(DEV), k_out=k, v_out=v)
        want = torch.full((T, 2 * H, D + 8), 9.0, dtype=torch.float16)
        ok = slots >= 0
        for a, x in ((0, vals[0]), (H, vals[1])):
            want[ok, a:a + H, shift:shift + D] = x[slots[ok] // 16, slots[ok] % 16].to(torch.float16)
        assert torch.equal(out.cpu(), want)


# ---------------------------------------------------------------- decode
def decode_case(ctx, G, H, D, BS, dtype, seed=0, hmaj=True, dual=False, sm_scale=None, amp=1.0, **kw):
    bt, P = R.tables(ctx, BS, seed=seed)
    cache, vals, tops = U.make_cache(pkv, P, BS, H, D, seed=seed, hmaj=hmaj, dual=dual, amp=amp)
    q = rand((len(ctx), H * G, D), seed + 1, dtype)
    sm = sm_scale if sm_scale is not None else D ** -0.5
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pkv.paged_decode(q.to(DEV), cache, bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV), sm_scale=sm, err_flag=err, **kw)
    torch.cuda.synchronize()
    assert err.item() == 0
    parts = U.decode_parts(q, vals, tops, bt, ctx, sm)
    U.close(out, parts, 15 * 0.3 * amp, dtype, D)
    return q, cache, vals, tops, bt, out, parts


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("BS", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("G,H,D", [(4, 8, 128), (1, 4, 128), (8, 2, 64), (5, 3, 64), (16, 4, 128), (9, 1, 64), (1, 1, 128), (7, 5, 128)])
def test_decode(dtype, BS, G, H, D):
    decode_case([1, 0, 15, 16, 17, 31, 32, 33, 64, 95, 130, 257], G, H, D, BS, dtype, seed=BS + G)


@pytest.mark.parametrize("G,H,D,BS", [(4, 8, 128, 16), (8, 8, 128, 32), (1, 32, 128, 16), (2, 6, 64, 64), (12, 8, 128, 32), (16, 2, 64, 16), (8, 1, 128, 32)])
def test_decode_of_long_contexts(G, H, D, BS):
    """Sequences over many CTAs and CTAs with many sequences."""
    decode_case([3000, 1, 0, 777, 5000, 64, 31], G, H, D, BS, torch.float16, seed=G)
    decode_case([1 + 37 * i % 211 for i in range(150)], G, H, D, BS, torch.bfloat16, seed=G + 1)


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("hmaj,dual", [(False, False), (True, True), (False, True)])
def test_decode_layouts_and_splits(splits, hmaj, dual):
    for BS in (16, 64):
        decode_case([5, 100, 333], 4, 6, 128, BS, torch.float16, hmaj=hmaj, dual=dual, num_splits=splits)


@pytest.mark.parametrize("sm", [-0.1, 0.0, 2.0, 1e-3])
def test_decode_softmax_scales(sm):
    for G in (2, 16):
        decode_case([1, 40, 200], G, 2, 128, 16, torch.float16, sm_scale=sm)


@pytest.mark.parametrize("amp", [2.0 ** -9, 2.0 ** 9])
def test_decode_scales_of_other_sizes(amp):
    """Small V scales keep their bits (weights times scales are packed to 16)."""
    bt, P = R.tables([300, 20], 16)
    cache, vals, tops = U.make_cache(pkv, P, 16, 2, 128)
    cache.v_qscale.mul_(amp)
    vals[1] = vals[1] * amp
    tops[1] = tops[1] * amp
    q = rand((2, 8, 128), 1, torch.bfloat16)
    ctx = [300, 20]
    out = pkv.paged_decode(q.to(DEV), cache, bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV))
    U.close(out, U.decode_parts(q, vals, tops, bt, ctx, 128 ** -0.5), 4.5 * amp, torch.bfloat16, 128)


def test_decode_v_scales_far_apart():
    """Each sequence's V scales between 2^-14 and 2^14: relative to the largest product."""
    ctx, BS = [70, 33, 200], 16
    bt, P = R.tables(ctx, BS)
    cache, vals, tops = U.make_cache(pkv, P, BS, 2, 128)
    e = torch.randint(-12, 12, (P, BS, 2), generator=torch.Generator().manual_seed(4))
    f = torch.ldexp(torch.ones(e.shape), e)
    cache.v_qscale.mul_(f.to(DEV).half())
    vals[1] = vals[1] * f.double()[..., None]
    tops[1] = tops[1] * f.double()[..., None]
    q = rand((3, 4, 128), 2, torch.float16, 0.2)
    out = pkv.paged_decode(q.to(DEV), cache, bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV))
    parts = U.decode_parts(q, vals, tops, bt, ctx, 128 ** -0.5)
    U.close(out, parts, 4.5 * 2.0 ** 11, torch.float16, 128)


@pytest.mark.parametrize("big", [2.0 ** 15, 2.0 ** -20, 3e30, 1e-30])
def test_decode_queries_of_any_size(big):
    """Queries are brought into f16's range by a power of two per row."""
    ctx = [90, 20]
    bt, P = R.tables(ctx, 32)
    cache, vals, tops = U.make_cache(pkv, P, 32, 2, 64)
    q = (rand((2, 6, 64), 3, torch.float32) * big).to(torch.bfloat16)
    q[:, 1] = rand((2, 64), 4, torch.bfloat16)             # another size in the same group
    sm = 0.125 / big if big > 1 else 0.125
    out = pkv.paged_decode(q.to(DEV), cache, bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV), sm_scale=sm)
    U.close(out, U.decode_parts(q, vals, tops, bt, ctx, sm), 4.5, torch.bfloat16, 64)


@pytest.mark.parametrize("BS", [8, 16, 32, 64])
def test_decode_ignores_what_is_behind_the_context(BS):
    ctx = [1, 17, 40, 75]
    bt, P = R.tables(ctx, BS)
    for G in (4, 12):
        cache, vals, tops = U.make_cache(pkv, P, BS, 2, 128)
        for b, c in enumerate(ctx):
            last = int(bt[b, (c - 1) // BS])
            for n in ("k_qscale", "v_qscale"):
                getattr(cache, n)[last, (c - 1) % BS + 1:] = float("nan")
                getattr(cache, n)[last, (c - 1) % BS + 2::2] = float("inf")
        q = rand((4, 2 * G, 128), 2, torch.float16)
        out = pkv.paged_decode(q.to(DEV), cache, bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV))
        U.close(out, U.decode_parts(q, vals, tops, bt, ctx, 128 ** -0.5), 4.5, torch.float16, 128)


def test_decode_zero_scales():
    """Rows of scale zero (constant rows) take part with the value zero."""
    ctx, BS = [50, 64], 16
    bt, P = R.tables(ctx, BS)
    cache, vals, tops = U.make_cache(pkv, P, BS, 1, 64)
    for i, (n, m) in enumerate((("k_qscale", 0), ("v_qscale", 1))):
        getattr(cache, n)[:, i::3] = 0
        vals[m][:, i::3] = 0
        tops[m][:, i::3] = 0
    q = rand((2, 4, 64), 2, torch.bfloat16)
    out = pkv.paged_decode(q.to(DEV), cache, bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV))
    U.close(out, U.decode_parts(q, vals, tops, bt, ctx, 0.125), 4.5, torch.bfloat16, 64)
    cache.v_qscale.zero_()
    out = pkv.paged_decode(q.to(DEV), cache, bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV))
    assert (out == 0).all()


@pytest.mark.parametrize("BS", [8, 16, 32, 64])
def test_decode_bad_tables(BS):
    """Blocks outside the pool are left out and flagged, lengths clamped."""
    ctx = [4 * BS, 3 * BS, 2 * BS + 5]
    bt, P = R.tables(ctx, BS, width=4)
    cache, vals, tops = U.make_cache(pkv, P, BS, 2, 128)
    q = rand((3, 8, 128), 2, torch.float16)
    bad = bt.clone()
    bad[0, 1], bad[2, 0] = P, -1
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pkv.paged_decode(q.to(DEV), cache, bad.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV), err_flag=err)
    assert err.item() == P_.DEVERR_BLOCK_RANGE
    # the tokens that are there, in a table without the bad blocks
    short = bt.clone()
    short[0, 1:3] = bt[0, 2:4]
    short[2, 0:2] = bt[2, 1:3]
    left = [3 * BS, 3 * BS, BS + 5]
    U.close(out, U.decode_parts(q, vals, tops, short, left, 128 ** -0.5), 4.5, torch.float16, 128)
    err.zero_()
    out = pkv.paged_decode(q.to(DEV), cache, bt.to(DEV), torch.tensor([-3, 1 << 30, 5], dtype=torch.int32, device=DEV), err_flag=err)
    assert err.item() & P_.DEVERR_CONTEXT_RANGE
    assert (out[0] == 0).all()


def test_decode_all_blocks_bad():
    cache, _, _ = U.make_cache(pkv, 2, 16, 1, 64)
    bt = torch.full((1, 4), -1, dtype=torch.int32, device=DEV)
    q = rand((1, 4, 64), 2, torch.float16).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pkv.paged_decode(q, cache, bt, torch.tensor([60], dtype=torch.int32, device=DEV), err_flag=err)
    assert err.item() == P_.DEVERR_BLOCK_RANGE and (out == 0).all()


def test_decode_strided_tensors():
    ctx, BS, H, G, D = [100, 30, 64], 16, 2, 4, 128
    bt, P = R.tables(ctx, BS)
    cache, vals, tops = U.make_cache(pkv, P, BS, H, D)
    q = rand((3, 2 * H * G, D), 2, torch.float16)
    wide = q.to(DEV)[:, ::2]
    out = torch.full((3, H * G, 2 * D), 9.0, dtype=torch.float16, device=DEV)
    cl = torch.tensor([[c, -9] for c in ctx], dtype=torch.int32, device=DEV)[:, 0]
    tab = torch.stack([bt, torch.full_like(bt, -9)], -1).to(DEV)[..., 0]
    pkv.paged_decode(wide, cache, tab, cl, out=out[..., 1:1 + D])
    parts = U.decode_parts(q[:, ::2], vals, tops, bt, ctx, D ** -0.5)
    U.close(out[..., 1:1 + D], parts, 4.5, torch.float16, D)
    assert (out[..., 0] == 9).all() and (out[..., 1 + D:] == 9).all()
    # q rows off the 16-byte boundary take the general kernel
    odd = torch.zeros((3, H * G, D + 1), dtype=torch.float16, device=DEV)
    odd[..., 1:] = wide
    got = pkv.paged_decode(odd[..., 1:], cache, tab, cl, out=torch.empty((3, H * G, D), dtype=torch.float16, device=DEV))
    U.close(got, parts, 4.5, torch.float16, D)


def test_decode_metadata_of_any_stride():
    ctx, BS, H, D = [100, 30], 16, 3, 64
    bt, P = R.tables(ctx, BS)
    cache, vals, tops = U.make_cache(pkv, P, BS, H, D, hmaj=False)
    for n in ("k_qscale", "v_qscale", "k_qzero", "v_qzero"):
        t = getattr(cache, n)
        wide = torch.zeros((P, BS, H, 3), dtype=t.dtype, device=DEV)
        wide[..., 1] = t
        setattr(cache, n, wide[..., 1])
    q = rand((2, 3 * H, D), 2, torch.bfloat16)
    out = pkv.paged_decode(q.to(DEV), cache, bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV))
    U.close(out, U.decode_parts(q, vals, tops, bt, ctx, 0.125), 4.5, torch.bfloat16, D)


def test_decode_captured_and_garbage_workspace():
    q, cache, vals, tops, bt, want, _ = decode_case([500, 33, 1, 90], 4, 2, 128, 16, torch.float16)
    qd, bd = q.to(DEV), bt.to(DEV)
    cl = torch.tensor([500, 33, 1, 90], dtype=torch.int32, device=DEV)
    ws = torch.full((pkv.decode_workspace_bytes(qd, cache, bd),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(qd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pkv.paged_decode(qd, cache, bd, cl, out=out, workspace=ws)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_decode(qd, cache, bd, cl, out=out, workspace=ws)
    for _ in range(3):
        out.fill_(7)
        g.replay()
        assert torch.equal(out, want)
    cl.copy_(torch.tensor([1, 0, 64, 90], dtype=torch.int32))
    g.replay()
    fresh = pkv.paged_decode(qd, cache, bd, cl)
    assert torch.equal(out, fresh)


def test_decode_no_sequences():
    cache, _, _ = U.make_cache(pkv, 2, 16, 2, 64)
    q = torch.zeros((0, 4, 64), dtype=torch.float16, device=DEV)
    out = pkv.paged_decode(q, cache, torch.zeros((0, 3), dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV))
    assert out.shape == q.shape


def test_decode_noalloc():
    q, cache, vals, tops, bt, _, parts = decode_case([500, 33, 1], 4, 2, 128, 16, torch.float16)
    out = pkv.paged_decode_noalloc(q.to(DEV), cache, bt.to(DEV), torch.tensor([500, 33, 1], dtype=torch.int32, device=DEV))
    U.close(out, parts, 4.5, torch.float16, 128)


@pytest.mark.parametrize("D,BS", [(128, 16), (64, 32)])
def test_blocks_beyond_four_gigabytes(D, BS):
    """The pool's far blocks: addresses beyond 2^32 bytes."""
    H, row = 8, D // 2
    P = (1 << 32) // (BS * H * row) + 40
    k = torch.zeros((P, BS, H, row), dtype=torch.uint8, device=DEV)
    v = torch.zeros_like(k)
    meta = [torch.zeros((P, H, BS), dtype=t, device=DEV).transpose(1, 2) for t in (torch.float16, torch.uint8, torch.float16, torch.uint8)]
    far = pkv.KVCache("u4", k, v, k_qscale=meta[0], k_qzero=meta[1], v_qscale=meta[2], v_qzero=meta[3])
    T = 100
    x, y = rand((T, H, D), 1, torch.float16).to(DEV), rand((T, H, D), 2, torch.float16).to(DEV)
    near = pkv.KVCache.allocate("u4", 40, BS, H, D)
    slots = torch.arange(T, device=DEV)
    first = P - 40
    pkv.kv_append(x, y, slots, near)
    pkv.kv_append(x, y, slots + first * BS, far)
    for a, b in zip(pkv.kv_gather(near, slots), pkv.kv_gather(far, slots + first * BS)):
        assert torch.equal(a, b)
    q = rand((1, 2 * H, D), 3, torch.float16).to(DEV)
    bt = torch.arange(T // BS + 1, dtype=torch.int32, device=DEV)[None]
    cl = torch.tensor([T], dtype=torch.int32, device=DEV)
    assert torch.equal(pkv.paged_decode(q, near, bt, cl), pkv.paged_decode(q, far, bt + first, cl))
    qs = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    assert torch.equal(pkv.paged_prefill(q, near, bt, qs, cl), pkv.paged_prefill(q, far, bt + first, qs, cl))


# ---------------------------------------------------------------- prefill
def prefill_case(new, ctx, G, H, D, BS, dtype, seed=0, hmaj=True, dual=False, sm_scale=None):
    bt, P = R.tables(ctx, BS, seed=seed)
    cache, vals, tops = U.make_cache(pkv, P, BS, H, D, seed=seed, hmaj=hmaj, dual=dual)
    starts = list(itertools.accumulate(new, initial=0))
    q = rand((starts[-1], H * G, D), seed + 1, dtype)
    sm = sm_scale if sm_scale is not None else D ** -0.5
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    out = pkv.paged_prefill(q.to(DEV), cache, bt.to(DEV), i32(starts), i32(ctx), sm_scale=sm, err_flag=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    parts = U.prefill_parts(q, vals, tops, bt, starts, ctx, sm)
    U.close(out, parts, 4.5, dtype, D)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("BS", [8, 16, 64, 256])
@pytest.mark.parametrize("G,H,D", [(4, 2, 128), (1, 4, 128), (3, 3, 64), (17, 1, 128)])
def test_prefill(dtype, BS, G, H, D):
    prefill_case([1, 0, 5, 130, 33], [1, 40, 5, 130, 400], G, H, D, BS, dtype, seed=G)


@pytest.mark.parametrize("hmaj,dual", [(False, False), (True, True)])
def test_prefill_layouts(hmaj, dual):
    prefill_case([3, 70, 260], [700, 70, 300], 4, 4, 128, 16, torch.float16, hmaj=hmaj, dual=dual)
    prefill_case([3, 70, 260], [700, 70, 300], 4, 4, 64, 32, torch.bfloat16, hmaj=hmaj, dual=dual, sm_scale=-0.07)


def test_prefill_ignores_hidden_scales():
    """Scales of tokens that a row does not see may be anything."""
    BS, H, D, n, c = 16, 2, 128, 20, 50
    bt, P = R.tables([c], BS)
    cache, vals, tops = U.make_cache(pkv, P, BS, H, D)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    q = rand((n, 4, D), 1, torch.float16)
    at = c - 5                                    # seen by the last five rows alone
    cache.v_qscale[int(bt[0, at // BS]), at % BS] = float("nan")
    last = int(bt[0, (c - 1) // BS])
    cache.k_qscale[last, (c - 1) % BS + 1:] = float("nan")
    out = pkv.paged_prefill(q.to(DEV), cache, bt.to(DEV), i32([0, n]), i32([c]))
    parts = U.prefill_parts(q, vals, tops, bt, [0, n], [c], D ** -0.5)
    assert out[n - 5:].isnan().all()
    U.close(out[:n - 5], tuple(t[:n - 5] for t in parts), 4.5, torch.float16, D)


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("BS,D", [(16, 128), (32, 64)])
def test_prompt_then_decode_steps(dtype, BS, D):
    """Prompts appended and attended, then decode steps of one call each,
    against attention over the rows as stored."""
    H, G, prompts, steps = 2, 4, [37, 5, 64], 3
    total = [n + steps for n in prompts]
    bt, P = R.tables(total, BS)
    cache = pkv.KVCache.allocate("u4", P, BS, H, D, fill=0xFF)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    btd = bt.to(DEV)

    def stored():
        slots = torch.arange(P * BS, device=DEV)
        v64 = []
        for d, s, z in ((cache.k_cache, cache.k_qscale, cache.k_qzero), (cache.v_cache, cache.v_qscale, cache.v_qzero)):
            c, sd, zd = U.numpy_codes(d).double(), s.cpu().double()[..., None], z.cpu().double()[..., None]
            v64.append(((c - zd) * sd, (c + zd) * sd))
        del slots
        return [v64[0][0], v64[1][0]], [v64[0][1], v64[1][1]]

    starts = list(itertools.accumulate(prompts, initial=0))
    T = starts[-1]
    k, v, q = rand((T, H, D), 1, dtype), rand((T, H, D), 2, dtype), rand((T, H * G, D), 3, dtype)
    req = torch.repeat_interleave(torch.arange(3), torch.tensor(prompts))
    pos = torch.cat([torch.arange(n) for n in prompts])
    slots = pkv.slot_mapping(btd, i32(req.tolist()), i32(pos.tolist()), BS)
    pkv.kv_append(k.to(DEV), v.to(DEV), slots, cache)
    out = pkv.paged_prefill(q.to(DEV), cache, btd, i32(starts), i32(prompts))
    vals, tops = stored()
    vals = [torch.nan_to_num(t) for t in vals]
    tops = [torch.nan_to_num(t) for t in tops]
    U.close(out, U.prefill_parts(q, vals, tops, bt, starts, prompts, D ** -0.5), 8.0, dtype, D)
    for step in range(steps):
        ctx = [n + step + 1 for n in prompts]
        k, v, q = rand((3, H, D), 10 + step, dtype), rand((3, H, D), 20 + step, dtype), rand((3, H * G, D), 30 + step, dtype)
        out = pkv.decode_step(k.to(DEV), v.to(DEV), i32([0, 1, 2]), i32([c - 1 for c in ctx]), q.to(DEV), cache, btd, i32(ctx))
        vals, tops = stored()
        vals = [torch.nan_to_num(t) for t in vals]
        tops = [torch.nan_to_num(t) for t in tops]
        U.close(out, U.decode_parts(q, vals, tops, bt, ctx, D ** -0.5), 8.0, dtype, D)
        # the newest row is what a plain append of it stores
        at = bt[torch.arange(3), (torch.tensor(ctx) - 1) // BS].long(), (torch.tensor(ctx) - 1) % BS
        codes, s, z = U.quantise(k)
        assert torch.equal(U.numpy_codes(cache.k_cache)[at], codes)
        assert torch.equal(cache.k_qscale.cpu()[at], s) and torch.equal(cache.k_qzero.cpu()[at], z)


def test_two_streams():
    """Calls with workspaces of their own on two streams at once."""
    a = decode_case([700, 80], 4, 2, 128, 16, torch.float16, seed=1)
    b = decode_case([300, 900], 8, 1, 64, 32, torch.bfloat16, seed=2)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    args = []
    for (q, cache, _, _, bt, want, _), ctx in ((a, [700, 80]), (b, [300, 900])):
        args.append((q.to(DEV), cache, bt.to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV), want))
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for s, (q, cache, bt, cl, _) in zip(streams, args):
            with torch.cuda.stream(s):
                outs.append(pkv.paged_decode(q, cache, bt, cl))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, args[i % 2][4])


def test_launch_counts():
    cache, _, _ = U.make_cache(pkv, 4, 16, 2, 128)
    q = torch.zeros((2, 4, 128), dtype=torch.float16, device=DEV)
    bt = torch.zeros((2, 4), dtype=torch.int32, device=DEV)
    assert pkv.decode_launches(q, cache, bt) == 2 and pkv.decode_launches(q, cache, bt, num_splits=1) == 1
