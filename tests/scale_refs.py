"""Caches of given codes and scales, and attention in float64 with what its
tolerances need where scales lie far apart."""
import math

import torch

from tests import prompt_refs as R

CMAX = {"e4m3": 448.0, "e5m2": 57344.0, "i8": 127.0, "u3": 7.0}


def codes_of(kind, shape, seed):
    """Random codes (as stored) and their values in float64; of 3-bit caches
    (codes, zero points, codes minus zero points)."""
    g = torch.Generator().manual_seed(seed)
    if kind == "u3":
        c = torch.randint(0, 8, shape, generator=g)
        z = torch.randint(2, 6, shape[:-1], generator=g)
        return c, z, (c - z[..., None]).double()
    if kind == "i8":
        c = torch.randint(-127, 128, shape, generator=g).to(torch.int8)
        return c, None, c.double()
    x = (torch.randn(shape, generator=g) * R.QMAX[kind] / 5).clamp(-R.QMAX[kind], R.QMAX[kind]).to(R.CODE[kind])
    return x.view(torch.uint8), None, x.double()


def coded_cache(pkv, kind, scales, ks, vs, D, layout="flash", seed=0, device="cuda"):
    """A cache of random codes with the given scales [P, BS, H] (per block:
    the same within one), and its values (k, v) in float64."""
    P, BS, H = ks.shape
    vals, halves = [], []
    for i, s in enumerate((ks, vs)):
        c, z, x = codes_of(kind, (P, BS, H, D), seed + i)
        if kind == "u3":
            s, c = s.to(torch.float16), torch.from_numpy(R.pack3(c.numpy()))
        else:
            s = s.float()
        vals.append(x * s.double()[..., None])
        hm = lambda t: t.transpose(1, 2).contiguous().to(device).transpose(1, 2)  # noqa: E731
        if layout == "xvec":
            c = R.to_xvec(c)
        halves.append((c.to(device), s[:, 0].contiguous().to(device) if scales == "block" else hm(s),
                       hm(z.to(torch.uint8)) if z is not None else None))
    (kd, ks, kz), (vd, vs, vz) = halves
    if kind == "u3":
        c = pkv.KVCache(kind, kd, vd, k_qscale=ks, k_qzero=kz, v_qscale=vs, v_qzero=vz)
    else:
        c = pkv.KVCache(kind, kd, vd, scale_mode=scales, k_scales=ks, v_scales=vs, layout=layout)
    return c, vals[0], vals[1]


def flat_scale(kind, shape, amp=1.0):
    """Scales under which rows of codes_of have an amplitude of about `amp`."""
    return torch.full(shape, amp * {"e4m3": 2.0 ** -7, "e5m2": 2.0 ** -14, "i8": 2.0 ** -6, "u3": 2.0 ** -1}[kind])


def lead(q, kv, vs, bt, q_starts, ctx, sm_scale, total=False):
    """The largest weight times V scale that each row sees, or their sum: [T, Hq]."""
    T, Hq, D = q.shape
    BS, H = kv.shape[1], kv.shape[2]
    out = torch.zeros((T, Hq), dtype=torch.float64)
    for b in range(len(ctx)):
        s0, s1, c = int(q_starts[b]), int(q_starts[b + 1]), int(ctx[b])
        n = s1 - s0
        if n == 0 or c == 0:
            continue
        pos = torch.arange(c)
        ids = bt[b].long()[pos // BS]
        s = torch.einsum("nhgd,chd->hgnc", q[s0:s1].double().view(n, H, Hq // H, D), kv[ids, pos % BS]) * sm_scale
        s = s.masked_fill(pos[None, :] > (c - n + torch.arange(n))[:, None], -math.inf)
        p = torch.nan_to_num(torch.softmax(s, -1), 0.0)
        w = p * vs.double()[ids, pos % BS].T[:, None, None, :]
        out[s0:s1] = (w.sum(-1) if total else w.amax(-1)).permute(2, 0, 1).reshape(n, Hq)
    return out


def tolerance(ref, top_term, kind, dtype, D):
    """R.prefill_tolerance, and what rounding the weights times V scales to f16
    adds where they are far below the row's largest such term L: they are held
    relative to at most 2^5 L, so one below 2^-14 of that is off by at most
    2^-25 of it, times its code, for each key."""
    o, mean, top, keys = ref
    tol = R.prefill_tolerance(o, mean, top, keys, 0.0, dtype, D)
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25          # an output below the normal range
    return tol + 2.0 ** -20 * top_term[..., None] * keys[:, None, None] * CMAX[kind]
