"""kv_append_dynamic (bit exact against its definition), kv_gather (exact
values), and the prompt path as a serving loop runs it: append, prefill,
read back."""
import pytest
import torch

from tests import prompt_refs as R

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_num_gb300 as P
    P.lib()
    return P


def rows(T, H, D, dtype, seed):
    """Rows with the values that casts get wrong: zeros, tiny and huge rows,
    infinities, NaN, quotients on the rounding borders."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, D), generator=g)
    x *= torch.exp2(torch.randint(-12, 6, (T, H, 1), generator=g).float())
    x = x.to(dtype)
    if T > 12:
        x[0] = 0
        x[1] = -0.0
        x[2, :, 5] = float("nan")
        x[3, :, 7] = float("inf")
        x[4, :, 9] = -float("inf")
        x[5] = float("nan")
        x[6] = float("inf")
        x[7] = torch.finfo(dtype).max
        x[8] = torch.finfo(dtype).smallest_normal * torch.randn((H, D), generator=g).to(dtype)
        # smallest subnormals of the type
        x[9] = (torch.randint(0, 5, (H, D), generator=g).to(torch.int16)).view(dtype)
        # eighths of the largest: quotients on ties
        x[10] = (torch.randint(-16, 17, (H, D), generator=g).float() / 16).to(dtype)
        x[10, :, 0] = 1.0
        x[11] = (torch.randint(-254, 255, (H, D), generator=g).float()).to(dtype)
        x[11, :, 0] = 254.0
    return x


def from_layout(t, layout):
    return t.permute(0, 3, 1, 2, 4).flatten(-2) if layout == "xvec" else t


@pytest.mark.parametrize("layout", ["flash", "xvec"])
@pytest.mark.parametrize("D,H", [(128, 8), (64, 5), (128, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2", "i8"])
def test_dynamic_append_is_exact(pkv, kind, dtype, D, H, layout):
    T, P, BS = 333, 30, 16
    k, v = rows(T, H, D, dtype, 1), rows(T, H, D, dtype, 2)
    slots = torch.randperm(P * BS, generator=torch.Generator().manual_seed(3))[:T]
    slots[20:30] = -1                                  # padding tokens
    cache = pkv.KVCache.allocate(kind, P, BS, H, D, fill=0x5A, scale_mode="token", layout=layout)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.kv_append_dynamic(k.to(DEV), v.to(DEV), slots.to(DEV), cache, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    live = slots >= 0
    for x, buf, sc in ((k, cache.k_cache, cache.k_scales), (v, cache.v_cache, cache.v_scales)):
        codes, s = R.dynamic_append(x, kind)
        want = torch.full((P * BS, H, D), 0x5A, dtype=codes.dtype)
        want[slots[live]] = codes[live]
        ws = torch.ones((P * BS, H))
        ws[slots[live]] = s[live]
        got = from_layout(buf, layout).cpu().reshape(P * BS, H, D)
        assert torch.equal(got, want)
        assert torch.equal(sc.cpu().reshape(P * BS, H), ws)
        assert (s >= 2.0 ** -126).all() and torch.isfinite(s).all()


@pytest.mark.parametrize("T", [1, 2, 7, 5000])
def test_dynamic_append_sizes_and_strides(pkv, T):
    """Rows from sources with strides, off the 16-byte boundary too; scales
    stored slot by slot."""
    H, D, BS = 3, 64, 32
    P = T // BS + 2
    for pad in (0, 3):
        wide = torch.randn((T, 2 * H, D + pad), generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).to(DEV)
        k, v = wide[:, 0::2, pad:], wide[:, 1::2, pad:]
        cache = pkv.KVCache.allocate("e4m3", P, BS, H, D, fill=0, scale_mode="token")
        cache.k_scales, cache.v_scales = torch.ones((2, P, BS, H), device=DEV)
        slots = torch.randperm(P * BS, generator=torch.Generator().manual_seed(4))[:T].to(DEV)
        pkv.kv_append_dynamic(k, v, slots, cache)
        for x, buf, sc in ((k, cache.k_cache, cache.k_scales), (v, cache.v_cache, cache.v_scales)):
            codes, s = R.dynamic_append(x.cpu(), "e4m3")
            assert torch.equal(buf.view(P * BS, H, D)[slots].cpu(), codes)
            assert torch.equal(sc.view(P * BS, H)[slots].cpu(), s)


def test_dynamic_equals_scaled_append(pkv):
    """kv_append_scaled with the scales that kv_append_dynamic stored writes the same codes."""
    T, H, D, P, BS = 200, 4, 128, 20, 16
    k, v = (torch.randn((T, H, D), generator=torch.Generator().manual_seed(i)).half().to(DEV) for i in (5, 6))
    slots = torch.randperm(P * BS, generator=torch.Generator().manual_seed(7))[:T].to(DEV)
    a = pkv.KVCache.allocate("i8", P, BS, H, D, fill=0, scale_mode="token")
    b = pkv.KVCache.allocate("i8", P, BS, H, D, fill=0, scale_mode="token")
    pkv.kv_append_dynamic(k, v, slots, a)
    ks, vs = (t.reshape(P * BS, H)[slots].contiguous() for t in (a.k_scales, a.v_scales))
    pkv.kv_append_scaled(k, v, ks, vs, slots, b)
    for x, y in zip(a.tensors(), b.tensors()):
        assert torch.equal(x, y)


def test_bad_slots_are_flagged(pkv):
    cache = pkv.KVCache.allocate("e4m3", 4, 16, 2, 64, fill=0, scale_mode="token")
    k = torch.randn((3, 2, 64), device=DEV).half()
    slots = torch.tensor([3, 64, 2 ** 40], device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.kv_append_dynamic(k, k, slots, cache, err_flag=err)
    assert int(err.item()) == pkv.pkv.DEVERR_SLOT_RANGE
    err.zero_()
    ko = torch.full((3, 2, 64), 9.0, dtype=torch.float16, device=DEV)
    vo = ko.clone()
    pkv.kv_gather(cache, slots, k_out=ko, v_out=vo, err_flag=err)
    assert int(err.item()) == pkv.pkv.DEVERR_SLOT_RANGE
    assert (ko[1:] == 9).all() and (vo[1:] == 9).all() and not (ko[0] == 9).all()


CACHES = [("bf16", "head", "flash"), ("f16", "head", "flash"), ("bf16", "head", "xvec"), ("e4m3", "head", "flash"),
          ("e4m3", "block", "flash"), ("e4m3", "token", "xvec"), ("e5m2", "head", "xvec"), ("e5m2", "token", "flash"),
          ("i8", "head", "flash"), ("i8", "block", "xvec"), ("i8", "token", "flash"), ("u3", "head", "flash")]


@pytest.mark.parametrize("D,H", [(128, 8), (64, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind,scales,layout", CACHES)
def test_gather_values(pkv, kind, scales, layout, dtype, D, H):
    """Every row read back is its value, rounded to fp32 and then to the
    output type; padding rows keep what they held; a slot read twice gives
    the same row twice."""
    P, BS, T = 9, 16, 100
    cache, kv, vv = R.make_cache(pkv, kind, P, BS, H, D, scales, layout, seed=31)
    slots = torch.randint(0, P * BS, (T,), generator=torch.Generator().manual_seed(32))
    slots[5] = slots[4]
    slots[10:13] = -1
    ko = torch.full((T, H, D), 3.0, dtype=dtype, device=DEV)
    vo = ko.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.kv_gather(cache, slots.to(DEV), k_out=ko, v_out=vo, err_flag=err)
    assert int(err.item()) == 0
    for out, val in ((ko, kv), (vo, vv)):
        want = val.view(P * BS, H, D)[slots.clamp(min=0)].float().to(dtype)
        want[slots < 0] = 3.0
        assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "u3"])
@pytest.mark.parametrize("T", [0, 1, 33, 4100])
def test_gather_sizes_and_strides(pkv, kind, T):
    """Lengths from nothing up; outputs with strides, off the 16-byte
    boundary too; slots with a stride; the allocating form."""
    H, D, BS = 5, 64, 8
    P = 70
    cache, kv, vv = R.make_cache(pkv, kind, P, BS, H, D, seed=33)
    slots = torch.randint(0, P * BS, (T, 2), generator=torch.Generator().manual_seed(34)).to(DEV)[:, 0]
    want = [x.view(P * BS, H, D)[slots.cpu()].float().to(torch.bfloat16) for x in (kv, vv)]
    for pad in (0, 3):
        buf = torch.full((T, 2 * H, D + pad), 8.0, dtype=torch.bfloat16, device=DEV)
        k, v = pkv.kv_gather(cache, slots, k_out=buf[:, 0::2, pad:], v_out=buf[:, 1::2, pad:])
        assert torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1])
        assert (buf[:, :, :pad] == 8).all()
    k, v = pkv.kv_gather(cache, slots)
    assert torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1])


def test_gather_of_special_codes(pkv):
    """NaN and infinity codes, and products beyond the output type's range."""
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(2, 2, 1, 64)
    one = torch.ones(1, device=DEV)
    for kind, dt in (("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)):
        cache = pkv.KVCache(kind, codes.to(DEV), codes.to(DEV), k_scale=one, v_scale=one * 1000)
        slots = torch.arange(4, device=DEV)
        k, v = pkv.kv_gather(cache, slots, dtype=torch.float16)
        x = codes.view(4, 1, 64).view(dt).float()
        for got, want in ((k, x.half()), (v, (x * 1000).half())):
            assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
            assert torch.equal(torch.nan_to_num(got.cpu(), 0.0), torch.nan_to_num(want, 0.0))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8", "u3"])
def test_prompt_path(pkv, kind):
    """A serving loop's prompt side: slots from positions, the prompt's rows
    appended (quantised on the way in), a first chunk and a second one
    attended, then one decode step, and the rows read back.  Each output is
    attention over what the cache holds, and what it holds is near the rows."""
    H, G, D, BS = 4, 4, 128, 16
    lens, cut = [150, 33, 260], [100, 33, 130]
    bt, P = R.tables([n + 1 for n in lens], BS, seed=35)
    g = torch.Generator().manual_seed(36)
    scales = "token" if kind in R.QMAX else "head"
    cache = pkv.KVCache.allocate(kind, P, BS, H, D, fill=0, scale_mode=scales)
    btd = bt.to(DEV)
    k_all = [torch.randn((n + 1, H, D), generator=g).bfloat16() for n in lens]
    v_all = [torch.randn((n + 1, H, D), generator=g).bfloat16() for n in lens]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def append(lo, hi):
        req = torch.cat([torch.full((b - a,), i, dtype=torch.int32) for i, (a, b) in enumerate(zip(lo, hi))]).to(DEV)
        pos = torch.cat([torch.arange(a, b, dtype=torch.int32) for a, b in zip(lo, hi)]).to(DEV)
        slots = pkv.slot_mapping(btd, req, pos, BS, err_flag=err)
        k = torch.cat([x[a:b] for x, a, b in zip(k_all, lo, hi)]).to(DEV)
        v = torch.cat([x[a:b] for x, a, b in zip(v_all, lo, hi)]).to(DEV)
        (pkv.kv_append_dynamic if scales == "token" else pkv.kv_append)(k, v, slots, cache, err_flag=err)
        return slots, k, v

    def attend(lo, hi):
        st = [0]
        for a, b in zip(lo, hi):
            st.append(st[-1] + b - a)
        q = torch.randn((st[-1], H * G, D), generator=g).bfloat16()
        out = pkv.paged_prefill(q.to(DEV), cache, btd, torch.tensor(st, dtype=torch.int32, device=DEV),
                                torch.tensor(hi, dtype=torch.int32, device=DEV), err_flag=err)
        return q, st, out

    def values():
        slots = torch.arange(P * BS, device=DEV)
        k, v = pkv.kv_gather(cache, slots, dtype=torch.bfloat16)
        return k, v

    zero = [0, 0, 0]
    append(zero, cut)
    q1, st1, o1 = attend(zero, cut)
    slots, k, v = append(cut, lens)
    q2, st2, o2 = attend(cut, lens)
    append(lens, [n + 1 for n in lens])
    q3, st3, o3 = attend(lens, [n + 1 for n in lens])
    dec = pkv.paged_decode(q3.to(DEV), cache, btd, torch.tensor([n + 1 for n in lens], dtype=torch.int32, device=DEV))
    kg, vg = pkv.kv_gather(cache, slots, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    # read back: within half a step of the code (e4m3 2^-4 of the value, or of
    # the smallest normal; int8 half of amax / 127; 3-bit 1.5 of (max - min) / 7) and of bf16
    for got, x in ((kg, k), (vg, v)):
        x, d = x.double(), (got.double() - x.double()).abs()
        top = x.abs().amax(-1, keepdim=True)
        code = {"bf16": 0 * x, "e4m3": torch.maximum(x.abs() * 2.0 ** -4, top / 448 * 2.0 ** -10),
                "i8": 0 * x + top / 127 / 2, "u3": 0 * x + 1.5 * (x.amax(-1, keepdim=True) - x.amin(-1, keepdim=True)) / 7}[kind]
        assert (d <= code * 1.001 + 2.0 ** -8 * got.double().abs()).all()
    # the attention is that of the values the cache holds.  They are read back
    # in bf16 (one more half step in each k and v), which the tolerance counts:
    # in a score, half a step of sum |q||k|
    kv, vv = (x.double().cpu().view(P, BS, H, D) for x in values())
    h = R.half_step(torch.bfloat16)
    for q, st, ctx, out in ((q1, st1, cut, o1), (q2, st2, lens, o2), (q3, st3, [n + 1 for n in lens], o3)):
        ref, mean, top, keys = R.prefill(q, kv, vv, bt, st, ctx, D ** -0.5)
        tol = R.prefill_tolerance(ref, mean, top, keys, float(vv.abs().max()), torch.bfloat16, D)
        if kind != "bf16":
            tol = tol + mean * (h + 2 * h * top[..., None])
        assert ((out.double().cpu() - ref).abs() <= tol).all()
    assert float((dec.double() - o3.double()).abs().max()) <= 8 * h * 4


def test_more_than_32_bits_of_bytes(pkv):
    """Gather and dynamic append at blocks beyond 2^32 bytes."""
    BS, H, D = 16, 8, 128
    P = (1 << 32) // (BS * H * D) + 8
    k = torch.zeros((P, BS, H, D), dtype=torch.uint8, device=DEV)
    v = torch.zeros((P, BS, H, D), dtype=torch.uint8, device=DEV)
    ks, vs = torch.ones((2, P, H, BS), device=DEV).transpose(2, 3)
    cache = pkv.KVCache("e4m3", k, v, scale_mode="token", k_scales=ks, v_scales=vs)
    x = torch.randn((50, H, D), generator=torch.Generator().manual_seed(37)).bfloat16()
    slots = torch.arange(P * BS - 50, P * BS, device=DEV)
    pkv.kv_append_dynamic(x.to(DEV), x.to(DEV), slots, cache)
    codes, s = R.dynamic_append(x, "e4m3")
    assert torch.equal(k.view(-1, H, D)[slots].cpu(), codes)
    ko, vo = pkv.kv_gather(cache, slots)
    want = (codes.view(torch.float8_e4m3fn).float() * s[..., None]).bfloat16()
    assert torch.equal(ko.cpu(), want) and torch.equal(vo.cpu(), want)


@pytest.mark.parametrize("dtype,bits", [(torch.bfloat16, 8), (torch.float16, 11)])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2", "i8"])
def test_dynamic_append_every_quotient(pkv, kind, dtype, bits):
    """Rows whose largest element has each significand, with every number of
    the type below it down to 2^-18 of it: the codes are those of the fp32
    division and the cast (as torch does them on the GPU)."""
    D, H, BS = 128, 8, 16
    tops = torch.arange(2 ** (bits - 1), 2 ** bits, device=DEV)
    if bits == 11:
        tops = tops[torch.randperm(tops.numel(), generator=torch.Generator(device=DEV).manual_seed(38), device=DEV)[:128]]
    mant = torch.arange(2 ** (bits - 1), 2 ** bits, device=DEV, dtype=torch.float32)
    x = torch.cat([mant * 2.0 ** -e for e in range(19)])                    # below 2^bits
    x = torch.cat([x, -x])
    x = torch.cat([x, x.new_zeros(-x.numel() % (D - 1))]).view(-1, D - 1)
    rows = torch.cat([x.new_zeros((x.shape[0], 1)), x], 1)                  # [R, D], the largest goes first
    all_rows = rows[None].expand(tops.numel(), -1, -1).clone()
    top = tops.float()[:, None, None]
    all_rows = torch.where(all_rows.abs() > top, torch.zeros_like(all_rows), all_rows)
    all_rows[:, :, 0] = top[:, :, 0]
    flat = (all_rows.view(-1, D) / 64).to(dtype)                            # exact: a power of two
    n = -(-flat.shape[0] // H) * H
    flat = torch.cat([flat, flat.new_zeros((n - flat.shape[0], D))])
    k = flat.view(-1, H, D)
    T = k.shape[0]
    cache = pkv.KVCache.allocate(kind, T // BS + 1, BS, H, D, fill=0, scale_mode="token")
    slots = torch.arange(T, device=DEV)
    pkv.kv_append_dynamic(k, k, slots, cache)
    a = k.float().abs().amax(-1)
    s = (a / torch.full((), R.QMAX[kind], device=DEV)).clamp(min=2.0 ** -126)
    y = k.float() / s[..., None]
    want = y.round().clamp(-127, 127).to(torch.int8) if kind == "i8" else \
        y.clamp(-R.QMAX[kind], R.QMAX[kind]).to(R.CODE[kind]).view(torch.uint8)
    got = cache.k_cache.view(-1, H, D)[:T]
    assert torch.equal(got, want)
    assert torch.equal(cache.v_cache.view(-1, H, D)[:T], want)
    assert torch.equal(cache.k_scales.reshape(-1, H)[:T], s)
