"""Plain 64-bit forms of the 4-bit cache: the rows' codes, caches with their
dequantised values, and one-token attention with its tolerance."""
import math

import numpy as np
import torch

from tests import prompt_refs as R


def pack4(codes):
    """[..., D] codes -> [..., D / 2] bytes: element d at bits 4d .. 4d + 3."""
    c = codes.to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def quantise(x):
    """Rows [..., D] (f16 / bf16, finite) -> (codes, scale f16, zero): lo =
    min(0, min), hi = max(0, max), s = f16((hi - lo) / 15) with 32-bit steps."""
    x = x.float()
    lo, hi = x.amin(-1, keepdim=True).clamp(max=0), x.amax(-1, keepdim=True).clamp(min=0)
    s = ((hi - lo) / torch.tensor(15.0)).to(torch.float16)
    s = torch.where(torch.isinf(s), torch.full_like(s, 65504.0), s).double()
    # a quotient of two fp32 numbers in float64, rounded to fp32, is the fp32 quotient
    step = lambda y: torch.where(s > 0, (y.double() / torch.where(s > 0, s, torch.ones_like(s))).float().round(), 0)  # noqa: E731
    z = step(-lo).clamp(0, 15)
    codes = torch.where(s > 0, (step(x) + z).clamp(0, 15), torch.zeros_like(x))
    return codes.to(torch.uint8), s[..., 0].to(torch.float16), z[..., 0].to(torch.uint8)


def store(t, device, hmaj=True):
    """[P, BS, H] scales or zeros on the device, head-major behind the view or as they are."""
    return t.transpose(1, 2).contiguous().to(device).transpose(1, 2) if hmaj else t.contiguous().to(device)


def make_cache(pkv, P, BS, H, D, seed=0, hmaj=True, device="cuda", dual=False, amp=1.0):
    """A u4 KVCache of random codes, and (k, v) values and their bounds (|u| +
    z) s, all float64 [P, BS, H, D] on the CPU."""
    g = torch.Generator().manual_seed(seed)
    data, meta, vals, tops = [], [], [], []
    for _ in range(2):
        codes = torch.randint(0, 16, (P, BS, H, D), generator=g)
        z = torch.randint(0, 16, (P, BS, H), generator=g).to(torch.uint8)
        s = (amp * (torch.rand((P, BS, H), generator=g) * 0.2 + 0.1)).to(torch.float16)
        data.append(pack4(codes))
        meta.append((store(s, device, hmaj), store(z, device, hmaj)))
        vals.append((codes.double() - z.double()[..., None]) * s.double()[..., None])
        tops.append((codes.double() + z.double()[..., None]) * s.double()[..., None])
    if dual:                                      # both halves of one [P, 2, H, BS, row] buffer
        both = torch.stack([d.transpose(1, 2) for d in data], 1).contiguous().to(device)
        kd, vd = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    else:
        kd, vd = (d.to(device) for d in data)
    (ks, kz), (vs, vz) = meta
    return pkv.KVCache("u4", kd, vd, k_qscale=ks, k_qzero=kz, v_qscale=vs, v_qzero=vz), vals, tops


def prefill_parts(q, vals, tops, bt, starts, ctx, sm_scale):
    """The definition in float64 and what its tolerance is made of: R.prefill's
    (out, mean |v|, error of a score, keys, mean (u + z) s of v).  The third is (D + 8)
    roundings of a step of 2^-23 (a tensor core's sums may cut instead of round) of the
    largest sum |q| (u + z) s, and, of kernels that take codes as f16 subnormals of
    2^-22, whose products are aligned as if they were 2^-14: a step of 2^-23 of |q|'s
    largest element, brought to at least 2^13, over 2^13 2^-22 for each of D / 16 + 1 sums
    of 16, that is 2^-14 of it times s."""
    out, mean, _, keys = R.prefill(q, vals[0], vals[1], bt, starts, ctx, sm_scale)
    T, Hq, D = q.shape
    H = vals[0].shape[2]
    top, wide = torch.zeros((T, Hq), dtype=torch.float64), torch.zeros_like(out)
    BS = vals[0].shape[1]
    for b in range(len(ctx)):
        s0, s1, c = int(starts[b]), int(starts[b + 1]), int(ctx[b])
        if s1 == s0 or c == 0:
            continue
        n = s1 - s0
        pos = torch.arange(c)
        ids = bt[b].long()[pos // BS]
        k, kt, vt = vals[0][ids, pos % BS], tops[0][ids, pos % BS], tops[1][ids, pos % BS]
        qb = q[s0:s1].double().view(n, H, Hq // H, D)
        seen = pos[None, :] <= (c - n + torch.arange(n))[:, None]
        s = (torch.einsum("nhgd,chd->hgnc", qb, k) * sm_scale).masked_fill(~seen, -math.inf)
        wide[s0:s1] = torch.einsum("hgnc,chd->nhgd", torch.nan_to_num(torch.softmax(s, -1)), vt).reshape(n, Hq, D)
        a = torch.einsum("nhgd,chd->hgnc", qb.abs(), kt) * abs(sm_scale)
        top[s0:s1] = (a * seen).amax(-1).permute(2, 0, 1).reshape(n, Hq)
    # a row of codes up to 15 has s = its largest (u + z) s over 15 at most
    cut = q.double().abs().amax(-1) * abs(sm_scale) * float(tops[0].max()) / 15
    return out, mean, (D + 8) * 2.0 ** -23 * top + (D / 16 + 1) * 2.0 ** -14 * cut, keys, wide


def tolerance(parts, vmax, dtype, D):
    """How far a kernel may be off that multiplies codes exactly, sums in fp32
    and rounds weights times V scales to f16 once:
      - the output's rounding, half a step of it;
      - the weights' rounding, half an f16 step each (2^-11 of the mean |v|);
      - the weights' error from the scores', in the weight and in the maximum, and exp2
        to 2^-21;
      - the sums over the keys of P u and P z, a step of 2^-23 a key of the mean (u + z) s,
        and, of codes taken as subnormals of 2^-22, a step of 2^-23 2^-14 over 2^-22, that is
        2^-15, of s = vmax / 15 and of the weights' largest of each 16 keys, together at most
        the weights' sum;
      - products P below f16's normal range, off by 2^-25 each where the largest is at
        least 2^-2: with u up to 15, and 15 s = vmax at most, 2^-23 vmax a key."""
    out, mean, score, keys, wide = parts
    h = R.half_step(dtype)
    keys = keys[:, None, None]
    tol = h * out.abs() * (1 + h) + mean * (2.0 ** -11 * (1 + h) + 2.0 ** -21 + 2 * score[..., None])
    tol = tol + wide * (keys + 8) * 2.0 ** -23 + (2.0 ** -15 / 15 + keys * 2.0 ** -23) * vmax
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    return tol + 1e-30


def decode_parts(q, vals, tops, bt, ctx, sm_scale):
    """One query token per sequence, as prefill_parts; an empty context gives zeros."""
    B = q.shape[0]
    starts = list(range(B + 1))
    parts = prefill_parts(q, vals, tops, bt, starts, [max(c, 1) for c in ctx], sm_scale)
    for b, c in enumerate(ctx):
        if c == 0:
            for t in parts:
                t[b] = 0
    return parts


def close(got, parts, vmax, dtype, D):
    tol = tolerance(parts, vmax, dtype, D)
    err = (got.double().cpu() - parts[0]).abs()
    worst = float((err / tol).max())
    assert worst <= 1.0, "%.3g times the tolerance (error %.3g)" % (worst, float(err.max()))


def numpy_codes(data):
    """[..., D / 2] bytes -> [..., D] codes."""
    b = data.cpu().numpy()
    return torch.from_numpy(np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1))
