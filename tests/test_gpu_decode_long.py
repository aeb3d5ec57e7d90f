"""Decode over long contexts of coded caches: the error of a whole row relative to
the row, where many keys have nearly the same weight and the output is small
against the sums that it is made of.

What a row of D elements may be off by, relative to its root mean square, V's
elements being independent and of mean zero (so that out is about sqrt(sum p^2) v):
  - the output's rounding and the weights' to 16 bits, uniform within half a step
    each: 1 / sqrt(3) of it, 0.75 with room for D = 64 elements, added as squares;
  - the scores', in the weight and in the sum of weights: D / 16 + 2 steps of the tensor
    core, each off by at most 2^-23 of the largest number in it: for int8 of 1279 times
    |q|'s sum (codes are code + 1152) times the scale; for 3-bit codes, which are
    subnormals whose products are aligned as if they were 2^-14, 2^-13 of |q|'s
    largest element times the scale; for the others of sum |q| |k|;
  - the sums over the keys, n / 8 steps, which may cut 2^-23 of the running sum
    each, exp2 to 2^-21."""
import pytest
import torch

import paged_kv_cache_num_gb300 as pkv
from tests import prompt_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "i8": torch.int8}


def filled(kind, n, P, BS, H, D, scales, layout, seed):
    """A cache of n appended normal rows, and its values [n, H, D] float64 on the device."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    k, v = (torch.randn((P * BS, H, D), generator=g, device=DEV).bfloat16() for _ in range(2))
    slots = torch.arange(P * BS, device=DEV)
    kw = {} if kind in ("u3", "bf16") else {"scale_mode": scales}
    cache = pkv.KVCache.allocate(kind, P, BS, H, D, layout=layout, **kw)
    if kind in ("u3", "bf16"):
        pkv.kv_append(k, v, slots, cache)
    elif scales == "token":
        pkv.kv_append_dynamic(k, v, slots, cache)
    else:
        cache.k_scale = cache.v_scale = torch.full((H,), 4.5 / R.QMAX[kind], device=DEV)
        pkv.kv_append(k, v, slots, cache)
    out = []
    for data, s3, z3, s1, st in ((cache.k_cache, cache.k_qscale, cache.k_qzero, cache.k_scale, cache.k_scales),
                                 (cache.v_cache, cache.v_qscale, cache.v_qzero, cache.v_scale, cache.v_scales)):
        if kind == "u3":
            b = data.reshape(P * BS, H, D // 8, 3).long()
            word = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
            codes = torch.stack([(word >> (3 * i)) & 7 for i in range(8)], -1).reshape(P * BS, H, D)
            x = (codes.double() - z3.reshape(P * BS, H, 1).double()) * s3.reshape(P * BS, H, 1).double()
        else:
            if layout == "xvec":
                data = data.permute(0, 3, 1, 2, 4).reshape(P, BS, H, D)
            x = (data if kind == "bf16" else data.view(CODES[kind])).double().reshape(P * BS, H, D)
            if kind != "bf16":
                x = x * (s1.double()[None, :, None] if scales == "head" else st.reshape(P * BS, H, 1).double())
        out.append(x[:n])
    return cache, out[0], out[1]


def long_case(kind, n, B, H, G, D, BS, amp, dtype, scales="head", layout="flash", seed=0):
    P = (n + BS - 1) // BS
    cache, kd, vd = filled(kind, n, P, BS, H, D, scales, layout, seed)
    q = (torch.randn((B, H * G, D), generator=torch.Generator(device=DEV).manual_seed(seed + 1), device=DEV) * amp).to(dtype)
    bt = torch.cat([torch.randperm(P - 1, generator=torch.Generator().manual_seed(seed)), torch.tensor([P - 1])]).to(torch.int32).to(DEV)
    cl = torch.full((B,), n, dtype=torch.int32, device=DEV)
    out = pkv.paged_decode(q, cache, bt[None].expand(B, P), cl)
    assert torch.equal(out, pkv.paged_decode(q, cache, bt[None].expand(B, P), cl))
    some = sorted({0, B // 2, B - 1})
    qs = q[some].double().view(len(some), H, G, D)
    s = torch.einsum("bhgd,nhd->bhgn", qs, kd) * D ** -0.5
    ref = torch.einsum("bhgn,nhd->bhgd", torch.softmax(s, -1), vd).reshape(len(some), H * G, D)
    err = (out[some].double() - ref).square().mean(-1).sqrt() / ref.square().mean(-1).sqrt()
    h = R.half_step(dtype)
    hp = R.half_step(torch.bfloat16 if kind == "bf16" else torch.float16)
    top = float(qs.abs().sum(-1).max())
    if kind == "i8":
        step = 2.0 ** -23 * 1279 * top * float((cache.k_scale if scales == "head" else cache.k_scales).max())
    elif kind == "u3":
        step = 2.0 ** -13 * float(q.abs().max()) * float(cache.k_qscale.max())
    else:
        step = 2.0 ** -23 * top * float(kd.abs().max())
    score = (D / 16 + 2) * step * D ** -0.5
    bound = 0.75 * (h * h + hp * hp) ** 0.5 + 2 * score + n / 8 * 2.0 ** -23 + 2.0 ** -21
    assert float(err.max()) <= bound, "relative error %.3g, bound %.3g" % (float(err.max()), bound)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("amp", [0.0, 0.5])
@pytest.mark.parametrize("B", [1, 300])
@pytest.mark.parametrize("kind", ["e4m3", "i8", "u3"])
def test_long_contexts(kind, dtype, amp, B):
    """A sequence over many CTAs, and CTAs that take whole sequences."""
    long_case(kind, 32768, B, 8, 4, 128, 32, amp, dtype)


@pytest.mark.parametrize("kind,n,B,H,G,D,BS,amp,dtype,scales,layout", [
    ("i8", 20000, 300, 8, 12, 128, 32, 0.5, torch.float16, "head", "flash"), ("i8", 16384, 200, 8, 4, 64, 16, 0.5, torch.float16, "head", "flash"),
    ("i8", 20000, 200, 8, 4, 128, 16, 0.0, torch.float16, "token", "flash"), ("i8", 16384, 200, 8, 8, 128, 32, 0.0, torch.float16, "head", "xvec"),
    ("i8", 30000, 60, 16, 1, 128, 64, 0.5, torch.bfloat16, "head", "flash"), ("e5m2", 16384, 200, 8, 8, 128, 32, 0.5, torch.float16, "head", "flash"),
    ("u3", 20000, 300, 8, 12, 128, 32, 0.0, torch.float16, "head", "flash"), ("u3", 20001, 300, 8, 4, 128, 16, 0.0, torch.float16, "head", "flash"),
    ("u3", 32768, 120, 16, 1, 128, 16, 0.0, torch.float16, "head", "flash"), ("u3", 32768, 120, 16, 1, 128, 32, 0.3, torch.bfloat16, "head", "flash"),
    ("u3", 32768, 200, 8, 2, 128, 64, 0.0, torch.float16, "head", "flash"), ("u3", 32700, 300, 3, 1, 128, 32, 0.0, torch.bfloat16, "head", "flash"),
    ("bf16", 20000, 200, 8, 4, 128, 32, 0.5, torch.bfloat16, "head", "flash")])
def test_long_contexts_of_other_shapes(kind, n, B, H, G, D, BS, amp, dtype, scales, layout):
    long_case(kind, n, B, H, G, D, BS, amp, dtype, scales, layout)
