"""paged_prefill of rows that see values that are not finite, where their keys
are shared out between the halves of a row tile and between CTAs: such a row
is not finite, however its keys are divided."""
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


def attend(pkv, q, cache, bt, new, ctx):
    st = [0]
    for n in new:
        st.append(st[-1] + n)
    dev = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (st, ctx)]
    return pkv.paged_prefill(q.to(DEV), cache, bt.to(DEV), *dev).cpu()


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("n", [1, 3, 8])
@pytest.mark.parametrize("ctx", [129, 257, 385, 2049])
def test_a_nan_key_alone_in_its_tile(pkv, kind, n, ctx):
    """The newest token's K row is NaN and the first of a key tile: the last
    new row sees it, the others do not."""
    H, G, D, BS = 2, 4, 128, 16
    bt, P = R.tables([ctx], BS, seed=ctx)
    cache, kv, vv = R.make_cache(pkv, kind, P, BS, H, D, seed=1)
    at = ctx - 1
    cache.k_cache[int(bt[0, at // BS]), at % BS] = 0x7F if kind == "e4m3" else float("nan")
    dt = torch.float16 if kind == "f16" else torch.bfloat16
    q = torch.randn((n, H * G, D), generator=torch.Generator().manual_seed(2)).to(dt)
    out = attend(pkv, q, cache, bt, [n], [ctx])
    assert torch.isnan(out[-1]).all() and torch.isfinite(out[:-1]).all()


@pytest.mark.parametrize("kind,scales", [("bf16", "head"), ("f16", "head"), ("e4m3", "head"), ("i8", "token"), ("u3", "head")])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("ctx", [40, 200, 300, 3000])
def test_a_nan_query_row(pkv, kind, scales, n, ctx):
    H, G, D, BS = 1, 4, 128, 16
    bt, P = R.tables([ctx], BS, seed=3)
    cache, kv, vv = R.make_cache(pkv, kind, P, BS, H, D, scales, seed=4)
    q = torch.randn((n, H * G, D), generator=torch.Generator().manual_seed(5)).to(torch.float16 if kind == "f16" else torch.bfloat16)
    q[n // 2, 1] = float("nan")
    out = attend(pkv, q, cache, bt, [n], [ctx])
    bad = torch.zeros((n, H * G), dtype=torch.bool)
    bad[n // 2, 1] = True
    assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad]).all()


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("ctx", [256, 300, 5000])
def test_a_part_of_no_weight(pkv, what, value, ctx):
    """The value that is not finite lies among keys whose weights are below
    the smallest number beside those of the last tile: the row sees it all
    the same."""
    H, G, D, BS = 1, 4, 128, 16
    bt, P = R.tables([ctx], BS, seed=6)
    cache, kv, vv = R.make_cache(pkv, "bf16", P, BS, H, D, seed=7)
    q = torch.randn((1, H * G, D), generator=torch.Generator().manual_seed(8)).abs().bfloat16()
    # keys of the last tile along the (positive) queries: scores of several hundred
    for t in range((ctx - 1) // 128 * 128, ctx):
        cache.k_cache[int(bt[0, t // BS]), t % BS] = 64.0
    buf = cache.k_cache if what == "k" else cache.v_cache
    buf[int(bt[0, 0]), 5, :, 9] = value
    if what == "v":                          # only its column is touched
        out = attend(pkv, q, cache, bt, [1], [ctx])
        assert not torch.isfinite(out[:, :, 9]).any()
        assert torch.isfinite(out[:, :, :9]).all() and torch.isfinite(out[:, :, 10:]).all()
    elif value != value:
        assert torch.isnan(attend(pkv, q, cache, bt, [1], [ctx])).all()
    else:                                    # a score of +infinity
        assert not torch.isfinite(attend(pkv, q, cache, bt, [1], [ctx])).any()


@pytest.mark.parametrize("what", ["k_scale", "v_scale"])
@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_a_nan_scale_of_a_head(pkv, kind, what):
    """Rows of that head's q heads are NaN, but for those that see no key."""
    H, G, D, BS, new, ctx = 2, 4, 128, 16, [40, 30, 150], [40, 5, 2000]
    bt, P = R.tables(ctx, BS, seed=9)
    cache, kv, vv = R.make_cache(pkv, kind, P, BS, H, D, seed=10)
    q = torch.randn((sum(new), H * G, D), generator=torch.Generator().manual_seed(11)).bfloat16()
    want = attend(pkv, q, cache, bt, new, ctx)
    getattr(cache, what)[1] = float("nan")
    out = attend(pkv, q, cache, bt, new, ctx)
    blind = slice(40, 40 + 25)
    assert torch.equal(out[:, :G], want[:, :G]) and (out[blind] == 0).all()
    sees = torch.ones(sum(new), dtype=torch.bool)
    sees[blind] = False
    assert torch.isnan(out[sees][:, G:]).all()
