"""Decode over 4-bit caches with long contexts: the error of a whole row relative
to the row, where many keys have nearly the same weight and the output is the
small difference of large sums.

What a row of D elements may be off by, relative to its root mean square, V's
elements being independent and of mean zero (so that out is about sqrt(sum p^2) v):
  - the output's rounding and the weights' to f16, uniform within half a step
    each: 1 / sqrt(3) of it, 0.75 with room for D = 64 elements, added as squares;
  - the scores': a step of 2^-23 of |q|'s largest element, brought to at least 2^13,
    over 2^13 2^-22 (codes as subnormals of 2^-22, whose products are aligned as if they
    were 2^-14), for each of D / 16 + 1 sums, times the largest scale; in the weight
    and in the sum of weights;
  - the sums over the keys, n / 8 steps of the tensor core, which may cut 2^-23 of
    the running sum each, exp2 to 2^-21."""
import pytest
import torch

import paged_kv_cache_num_gb300 as pkv
from tests import prompt_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def values(data, scale, zero):
    """[P, BS, H, D] float64 on the device."""
    codes = torch.stack([data & 15, data >> 4], -1).flatten(-2).double()
    return (codes - zero.double()[..., None]) * scale.double()[..., None]


def long_case(n, B, H, G, D, BS, amp, dtype, seed=0):
    P = (n + BS - 1) // BS
    g = torch.Generator(device=DEV).manual_seed(seed)
    k = torch.randn((P * BS, H, D), generator=g, device=DEV).half()
    v = torch.randn((P * BS, H, D), generator=g, device=DEV).half()
    cache = pkv.KVCache.allocate("u4", P, BS, H, D)
    pkv.kv_append(k, v, torch.arange(P * BS, device=DEV), cache)
    kd = values(cache.k_cache, cache.k_qscale, cache.k_qzero).flatten(0, 1)[:n]
    vd = values(cache.v_cache, cache.v_qscale, cache.v_qzero).flatten(0, 1)[:n]
    q = (torch.randn((B, H * G, D), generator=g, device=DEV) * amp).to(dtype)
    # every sequence has the same blocks, all but the last in another order than the pool's
    bt = torch.cat([torch.randperm(P - 1, generator=torch.Generator().manual_seed(seed)), torch.tensor([P - 1])]).to(torch.int32).to(DEV)
    cl = torch.full((B,), n, dtype=torch.int32, device=DEV)
    out = pkv.paged_decode(q, cache, bt[None].expand(B, P), cl)
    again = pkv.paged_decode(q, cache, bt[None].expand(B, P), cl)
    assert torch.equal(out, again)
    some = sorted({0, B // 2, B - 1})
    s = torch.einsum("bhgd,nhd->bhgn", q[some].double().view(len(some), H, G, D), kd) * D ** -0.5
    ref = torch.einsum("bhgn,nhd->bhgd", torch.softmax(s, -1), vd).reshape(len(some), H * G, D)
    err = (out[some].double() - ref).square().mean(-1).sqrt() / ref.square().mean(-1).sqrt()
    h = R.half_step(dtype)
    score = (D / 16 + 1) * 2.0 ** -14 * float(q.abs().max()) * float(cache.k_qscale.max()) * D ** -0.5
    bound = 0.75 * (h * h + 2.0 ** -22) ** 0.5 + 2 * score + n / 8 * 2.0 ** -23 + 2.0 ** -21
    assert float(err.max()) <= bound, "relative error %.3g, bound %.3g" % (float(err.max()), bound)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("amp", [0.0, 1.0])
@pytest.mark.parametrize("B", [1, 300])
def test_long_contexts(dtype, amp, B):
    """A sequence over many CTAs, and CTAs that take whole sequences."""
    long_case(32768, B, 8, 4, 128, 32, amp, dtype)


@pytest.mark.parametrize("n,B,H,G,D,BS,amp,dtype", [
    (20000, 300, 8, 8, 64, 16, 0.3, torch.float16), (16384, 320, 4, 16, 128, 64, 0.5, torch.float16), (30000, 200, 6, 1, 128, 16, 1.0, torch.float16),
    (32760, 330, 4, 12, 64, 32, 0.0, torch.bfloat16), (60001, 256, 8, 2, 128, 128, 0.0, torch.float16), (17, 3, 2, 4, 128, 16, 0.0, torch.float16)])
def test_long_contexts_of_other_shapes(n, B, H, G, D, BS, amp, dtype):
    long_case(n, B, H, G, D, BS, amp, dtype)
