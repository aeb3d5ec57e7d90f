"""Plain 64-bit forms of the prompt-side operators (prefill attention, append
with computed scales, gather), and caches with their dequantised values, made
on the CPU with torch and numpy."""
import math

import numpy as np
import torch

QMAX = {"e4m3": 448.0, "e5m2": 57344.0, "i8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "i8": torch.int8}
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype):
    """A rounding to `dtype` is off by at most this, relative to the value."""
    return torch.finfo(dtype).eps / 2


def pack3(codes):
    """[..., D] codes -> [..., 3 D / 8] bytes."""
    bits = ((codes[..., None].astype(np.uint8) >> np.arange(3, dtype=np.uint8)) & 1).reshape(*codes.shape[:-1], -1)
    return np.packbits(bits, axis=-1, bitorder="little")


def to_xvec(t):
    """[P, BS, H, D] -> [P, H, D / x, BS, x]."""
    P, BS, H, D = t.shape
    x = 16 // t.element_size()
    return t.reshape(P, BS, H, D // x, x).permute(0, 2, 3, 1, 4).contiguous()


def make_cache(pkv, kind, P, BS, H, D, scales="head", layout="flash", seed=0, dual=False, device="cuda", amp=1.0):
    """A KVCache of random rows on `device`, and its values (k, v) in float64
    [P, BS, H, D] on the CPU."""
    g = torch.Generator().manual_seed(seed)
    vals, halves = [], []
    for _ in range(2):
        if kind == "u3":
            codes = torch.randint(0, 8, (P, BS, H, D), generator=g)
            z = torch.randint(0, 8, (P, BS, H), generator=g).to(torch.uint8)
            s = (amp * (torch.rand((P, BS, H), generator=g) * 0.5 + 0.25)).to(torch.float16)
            data = torch.from_numpy(pack3(codes.numpy()))
            vals.append((codes.double() - z.double()[..., None]) * s.double()[..., None])
            hm = lambda t: t.transpose(1, 2).contiguous().to(device).transpose(1, 2)  # noqa: E731
            halves.append((data, hm(s), hm(z)))
            continue
        x = torch.randn((P, BS, H, D), generator=g) * amp
        if kind in DT:
            data = x.to(DT[kind])
            vals.append(data.double())
            halves.append((data, None, None))
            continue
        if scales == "head":
            s = x.abs().amax((0, 1, 3)) / QMAX[kind]
            sc = s.view(1, 1, H, 1)
        elif scales == "block":
            s = x.abs().amax((1, 3)) / QMAX[kind] * (1 + torch.rand((P, H), generator=g))
            sc = s.view(P, 1, H, 1)
        else:
            s = x.abs().amax(3) / QMAX[kind]
            sc = s[..., None]
        y = x / sc
        data = y.round().clamp(-127, 127).to(torch.int8) if kind == "i8" else \
            y.clamp(-QMAX[kind], QMAX[kind]).to(CODE[kind])
        vals.append(data.double() * sc.double())
        data = data if kind == "i8" else data.view(torch.uint8)
        if scales == "token":
            s = s.transpose(1, 2).contiguous().to(device).transpose(1, 2)
        halves.append((data, s.to(device), None))
    (kd, ks, kz), (vd, vs, vz) = halves
    if layout == "xvec":
        kd, vd = to_xvec(kd).to(device), to_xvec(vd).to(device)
    elif dual:                                    # both halves of one [P, 2, H, BS, row] buffer
        both = torch.stack([kd.transpose(1, 2), vd.transpose(1, 2)], 1).contiguous().to(device)
        kd, vd = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    else:
        kd, vd = kd.to(device), vd.to(device)
    if kind == "u3":
        c = pkv.KVCache(kind, kd, vd, k_qscale=ks, k_qzero=kz, v_qscale=vs, v_qzero=vz)
    elif kind in DT:
        c = pkv.KVCache(kind, kd, vd, layout=layout)
    elif scales == "head":
        c = pkv.KVCache(kind, kd, vd, k_scale=ks, v_scale=vs, layout=layout)
    else:
        c = pkv.KVCache(kind, kd, vd, scale_mode=scales, k_scales=ks, v_scales=vs, layout=layout)
    return c, vals[0], vals[1]


def tables(ctx, BS, extra=3, seed=0, width=None):
    """(block_tables int32 [B, max], number of blocks): a random permutation
    of the pool; entries behind a sequence's last block are -7 (never read)."""
    need = [-(-max(t, 0) // BS) for t in ctx]
    P = sum(need) + extra
    ids = np.random.RandomState(seed).permutation(P)
    bt = np.full((len(ctx), width or max(1, max(need))), -7, np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
    return torch.from_numpy(bt), P


def prefill(q, kv, vv, bt, q_starts, ctx, sm_scale):
    """The definition in float64: (out, tol-ingredients).  q [T, Hq, D] any
    float type; kv / vv [P, BS, H, D] float64.  Returns out [T, Hq, D] and
    (mean |v| under the weights [T, Hq, D], largest |q|.|k| sum [T, Hq],
    number of keys [T]); rows that no sequence owns hold NaN."""
    T, Hq, D = q.shape
    BS, H = kv.shape[1], kv.shape[2]
    G = Hq // H
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.float64)
    mean, top = torch.zeros_like(out), torch.zeros((T, Hq), dtype=torch.float64)
    keys = torch.zeros(T, dtype=torch.float64)
    for b in range(len(ctx)):
        s0, s1 = int(q_starts[b]), int(q_starts[b + 1])
        n, c = s1 - s0, int(ctx[b])
        if n == 0:
            continue
        pos = torch.arange(c)
        ids = bt[b].long()[pos // BS]
        k, v = kv[ids, pos % BS], vv[ids, pos % BS]                # [c, H, D]
        qb = q[s0:s1].double().view(n, H, G, D)
        s = torch.einsum("nhgd,chd->hgnc", qb, k) * sm_scale
        a = torch.einsum("nhgd,chd->hgnc", qb.abs(), k.abs()) * abs(sm_scale)
        seen = pos[None, :] <= (c - n + torch.arange(n))[:, None]  # [n, c]
        s = s.masked_fill(~seen, -math.inf)
        m = s.amax(-1, keepdim=True) if c else torch.zeros((H, G, n, 1), dtype=torch.float64)
        p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
        l = p.sum(-1, keepdim=True)
        p = torch.where(l > 0, p / torch.where(l > 0, l, torch.ones_like(l)), torch.zeros_like(p))
        # a weight of zero times a value that is not finite is no part of the sum
        out[s0:s1] = torch.einsum("hgnc,chd->nhgd", p, torch.nan_to_num(v, 0, 0, 0)).reshape(n, Hq, D)
        mean[s0:s1] = torch.einsum("hgnc,chd->nhgd", p, torch.nan_to_num(v, 0, 0, 0).abs()).reshape(n, Hq, D)
        if c:
            top[s0:s1] = (a * seen).amax(-1).permute(2, 0, 1).reshape(n, Hq)
        keys[s0:s1] = seen.sum(-1).double()
    return out, mean, top, keys


def prefill_tolerance(out, mean, top, keys, vmax, dtype, D):
    """How far a kernel may be off that takes the products in 16-bit operands
    with fp32 sums: the final rounding (half a step of out), the weights'
    rounding to 16 bits (half a step each, so half a step of the mean |v|),
    the scores' fp32 sums (D + 3 roundings of 2^-24 of sum |q||k|, twice: in
    the weight and in the maximum), exp2 to 2^-21, the fp32 sums over the
    keys, and for f16 weights below the normal range (off by 2^-25 of a
    weight up to one, n of them; outputs below it likewise)."""
    h = half_step(dtype)
    fp32 = 2.0 ** -21 + 2 * (D + 3) * 2.0 ** -24 * top[..., None] + (keys[:, None, None] + 4) * 2.0 ** -23
    tol = h * out.abs() * (1 + h) + mean * (h * (1 + h) + fp32)
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25 * (1 + keys[:, None, None] * vmax)
    return tol + 1e-30


def dynamic_append(x, kind):
    """(codes, scales) of rows x [T, H, D] (f16 / bf16): the scale a / qmax
    in fp32 but at least 2^-126, the quotient in fp32, then the cast."""
    xd = x.double()
    fin = torch.where(torch.isfinite(xd), xd.abs(), torch.zeros_like(xd))
    # a quotient of two fp32 numbers in float64, rounded to fp32, is the fp32 quotient
    s = (fin.amax(-1) / QMAX[kind]).float().clamp(min=2.0 ** -126)
    y = (xd / s.double()[..., None]).float()
    if kind == "i8":
        return torch.nan_to_num(y, 0.0, 127.0, -127.0).double().round().clamp(-127, 127).to(torch.int8), s
    c = torch.nan_to_num(y, 0.0, QMAX[kind], -QMAX[kind]).clamp(-QMAX[kind], QMAX[kind]).to(CODE[kind]).view(torch.uint8)
    return torch.where(torch.isnan(y), torch.full_like(c, 0x7F), c), s
