"""paged_prefill in forms off the usual path: groups of more than 128 q heads
(a token's heads in several subtiles, Q by copies), and softmax scales below
zero over every kind of cache and strided queries."""
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


def run(pkv, kind, dtype, new, ctx, H, G, D=128, scales="head", layout="flash", sm_scale=None, strided=False, seed=0):
    BS = 16
    bt, P = R.tables(ctx, BS, seed=seed)
    cache, kv, vv = R.make_cache(pkv, kind, P, BS, H, D, scales, layout, seed=seed)
    st = [0]
    for n in new:
        st.append(st[-1] + n)
    wide = torch.randn((st[-1], H * G + 1, D + 8), generator=torch.Generator().manual_seed(seed + 1)).to(R.DT[dtype]).to(DEV)
    q = wide[:, 1:, :D] if strided else wide[:, 1:, :D].contiguous()
    scale = D ** -0.5 if sm_scale is None else sm_scale
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dev = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (st, ctx)]
    out = pkv.paged_prefill(q, cache, bt.to(DEV), *dev, sm_scale=scale, err_flag=err)
    assert int(err.item()) == 0
    ref = R.prefill(q.cpu(), kv, vv, bt, st, ctx, scale)
    tol = R.prefill_tolerance(*ref, float(vv.abs().max()), R.DT[dtype], D)
    d = (out.double().cpu() - ref[0]).abs()
    assert torch.isfinite(tol).all() and (d <= tol).all(), "worst %g of its tolerance" % float((d / tol).max())


@pytest.mark.parametrize("kind,dtype", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("i8", "f16"), ("u3", "bf16")])
@pytest.mark.parametrize("G", [96, 128, 129, 160, 300])
def test_large_groups(pkv, kind, dtype, G):
    run(pkv, kind, dtype, new=[3, 1, 20], ctx=[3, 200, 330], H=1, G=G, seed=G)


@pytest.mark.parametrize("layout", ["flash", "xvec"])
def test_large_groups_of_two_heads(pkv, layout):
    run(pkv, "bf16", "bf16", new=[2, 5], ctx=[300, 700], H=2, G=200, D=64, layout=layout, strided=True, seed=1)


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind,dtype,scales,layout",
                         [("bf16", "bf16", "head", "flash"), ("f16", "f16", "head", "xvec"), ("e4m3", "bf16", "head", "flash"),
                          ("e4m3", "f16", "token", "flash"), ("e5m2", "bf16", "block", "xvec"), ("i8", "bf16", "token", "flash"),
                          ("i8", "f16", "head", "xvec"), ("u3", "bf16", "head", "flash"), ("u3", "f16", "head", "flash")])
def test_negative_scale(pkv, kind, dtype, scales, layout, D, strided):
    run(pkv, kind, dtype, new=[140, 1, 30], ctx=[140, 400, 300], H=2, G=3, D=D, scales=scales, layout=layout,
        sm_scale=-0.07, strided=strided, seed=2)
