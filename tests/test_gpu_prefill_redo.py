"""paged_prefill where V holds NaN or infinities among the tokens that some
rows of a tile do not see: in tiles of a CTA of its own, in tiles joined from
several CTAs, and in calls of a single key tile."""
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


POISON = {"bf16": float("nan"), "f16": float("inf"), "e4m3": 0x7F, "e5m2": 0x7C}


def run(pkv, kind, new, ctx, at, cols, H=2, G=4, D=128, BS=16, scales="head", unaligned=False):
    """Token at[b] of sequence b has `cols` of its V row poisoned: rows before
    it are right, rows that see it not finite in those columns and right in
    the others."""
    bt, P = R.tables(ctx, BS, seed=1)
    cache, kv, vv = R.make_cache(pkv, kind, P, BS, H, D, scales, seed=2)
    for b, a in enumerate(at):
        if a is not None:
            cache.v_cache[int(bt[b, a // BS]), a % BS, :, cols] = POISON[kind]
    dt = torch.float16 if kind == "f16" else torch.bfloat16
    st = [0]
    for n in new:
        st.append(st[-1] + n)
    q = torch.randn((st[-1], H * G, D), generator=torch.Generator().manual_seed(3)).to(dt)
    dev = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (st, ctx)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.empty((st[-1], H * G, D + 1), dtype=dt, device=DEV)[..., 1:] if unaligned else None
    out = pkv.paged_prefill(q.to(DEV), cache, bt.to(DEV), *dev, out=out, err_flag=err).cpu()
    assert int(err.item()) == 0
    ref = R.prefill(q, kv, vv, bt, st, ctx, D ** -0.5)
    tol = R.prefill_tolerance(*ref, float(vv.abs().max()), dt, D)
    hit = torch.zeros(out.shape, dtype=torch.bool)
    for b, a in enumerate(at):
        if a is not None:
            first = max(0, a - (ctx[b] - new[b]))
            hit[st[b] + first:st[b + 1], :, cols] = True
    # a rounding of the poisoned row's other columns' sum is the same as without it
    assert not torch.isfinite(out[hit]).any()
    d = (out.double() - ref[0]).abs()
    assert torch.isfinite(out[~hit]).all() and (d <= tol)[~hit].all()


ALL, ONE = slice(None), slice(77, 78)


@pytest.mark.parametrize("cols", [ALL, ONE], ids=["row", "column"])
@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3", "e5m2"])
def test_joined_tiles(pkv, kind, cols):
    run(pkv, kind, [300, 5], [9000, 7001], [8850, 6999], cols)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind,scales", [("bf16", "head"), ("e4m3", "head"), ("e4m3", "token"), ("e5m2", "block")])
def test_whole_tiles(pkv, kind, scales, D):
    n = 60
    g = torch.Generator().manual_seed(4)
    new = torch.randint(130, 400, (n,), generator=g).tolist()
    at = [None if i % 3 == 0 else (x * (i % 7)) // 7 for i, x in enumerate(new)]
    run(pkv, kind, new, new, at, slice(33, 34), D=D, scales=scales)


def test_one_key_tile(pkv):
    run(pkv, "bf16", [100, 3], [100, 128], [57, 126], ONE)


def test_unaligned_out(pkv):
    run(pkv, "bf16", [300, 150], [3000, 150], [2801, 70], ONE, unaligned=True)


def test_every_row(pkv):
    """V is NaN in one column everywhere: that column is NaN, the others right."""
    H, G, D, BS, new, ctx = 2, 4, 128, 16, [900, 40], [900, 5000]
    bt, P = R.tables(ctx, BS, seed=5)
    cache, kv, vv = R.make_cache(pkv, "bf16", P, BS, H, D, seed=6)
    cache.v_cache[..., 5] = float("nan")
    st = [0, 900, 940]
    q = torch.randn((940, H * G, D), generator=torch.Generator().manual_seed(7)).bfloat16()
    dev = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (st, ctx)]
    out = pkv.paged_prefill(q.to(DEV), cache, bt.to(DEV), *dev).cpu()
    assert torch.isnan(out[..., 5]).all()
    ref = R.prefill(q, kv, vv, bt, st, ctx, D ** -0.5)
    d = (out.double() - ref[0]).abs() <= R.prefill_tolerance(*ref, 0.0, torch.bfloat16, D)
    d[..., 5] = True
    assert d.all()


def test_long_context(pkv):
    """A NaN late in a context of 150000 tokens: rows before it are right, and
    the call ends without an error."""
    H, G, D, BS, n, c, at = 1, 2, 64, 64, 200, 150000, 149850
    bt, P = R.tables([c], BS, seed=8)
    cache, kv, vv = R.make_cache(pkv, "bf16", P, BS, H, D, seed=9)
    cache.v_cache[int(bt[0, at // BS]), at % BS] = float("nan")
    q = torch.randn((n, H * G, D), generator=torch.Generator().manual_seed(10)).bfloat16()
    dev = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, n], [c])]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pkv.paged_prefill(q.to(DEV), cache, bt.to(DEV), *dev, err_flag=err).cpu()
    assert int(err.item()) == 0
    first = at - (c - n)
    assert torch.isnan(out[first:]).all()
    ref = tuple(x[:first] for x in R.prefill(q[:first], kv, vv, bt, [0, first], [at], D ** -0.5))
    d = (out[:first].double() - ref[0]).abs()
    assert (d <= R.prefill_tolerance(*ref, 0.0, torch.bfloat16, D)).all()


def test_replayed(pkv):
    """The marks of one call are no matter of the next: a workspace is used
    again after a call with NaN in V, in a graph."""
    H, G, D, BS, new, ctx = 2, 4, 128, 16, [300, 40], [300, 3000]
    bt, P = R.tables(ctx, BS, seed=11)
    cache, kv, vv = R.make_cache(pkv, "bf16", P, BS, H, D, seed=12)
    st = [0, 300, 340]
    q = torch.randn((340, H * G, D), generator=torch.Generator().manual_seed(13)).bfloat16().to(DEV)
    args = (bt.to(DEV), *(torch.tensor(x, dtype=torch.int32, device=DEV) for x in (st, ctx)))
    want = pkv.paged_prefill(q, cache, *args)
    ws = torch.empty(pkv.prefill_workspace_bytes(q, cache, args[0]), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_prefill(q, cache, *args, out=out, workspace=ws)
    place = int(bt[0, 200 // BS]), 200 % BS
    good = cache.v_cache[place].clone()
    for poisoned in (False, True, False, True, False):
        cache.v_cache[place] = float("nan") if poisoned else good
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        if not poisoned:
            assert torch.equal(out, want)
        else:
            assert torch.isnan(out[200:300]).all()
            assert torch.isfinite(out[:200]).all() and torch.equal(out[300:], want[300:])
