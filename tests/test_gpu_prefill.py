"""paged_prefill against attention in float64: every cache kind, layout and
scale granularity, packed sequences from one token up, contexts longer and
shorter than the new tokens, odd sizes and strides, masked places that hold
NaN, bad table data, rows that no sequence owns."""
import math

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


def starts_of(new, first=0):
    s = [first]
    for n in new:
        s.append(s[-1] + n)
    return s


def check(out, ref, dtype, D, vmax):
    o, mean, top, keys = ref
    owned = ~torch.isnan(o[:, 0, 0])
    tol = R.prefill_tolerance(o, mean, top, keys, vmax, dtype, D)
    d = (out.double().cpu() - o).abs()[owned]
    assert torch.isfinite(out[owned.to(out.device)]).all()
    bad = d > tol[owned]
    assert not bad.any(), "worst %g of its tolerance" % float((d / tol[owned]).max())
    # a few percent of the tolerance on average: a wrong mask or a lost key is not hidden by it
    assert float((d / tol[owned]).mean()) < 0.5


def case(pkv, kind, dtype, new, ctx, H=2, G=4, D=128, BS=16, scales="head", layout="flash", seed=0, sm_scale=None,
         dual=False, tail=0, amp=1.0):
    """Runs one call and compares it; returns what it used."""
    bt, P = R.tables(ctx, BS, seed=seed)
    cache, kv, vv = R.make_cache(pkv, kind, P, BS, H, D, scales, layout, seed=seed, dual=dual, amp=amp)
    g = torch.Generator().manual_seed(seed + 1)
    st = starts_of(new)
    q = torch.randn((st[-1] + tail, H * G, D), generator=g).to(R.DT[dtype])
    scale = 1 / math.sqrt(D) if sm_scale is None else sm_scale
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (q.to(DEV), cache, bt.to(DEV), torch.tensor(st, dtype=torch.int32, device=DEV),
            torch.tensor(ctx, dtype=torch.int32, device=DEV))
    out = pkv.paged_prefill(*args, sm_scale=scale, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(out, R.prefill(q, kv, vv, bt, st, ctx, scale), R.DT[dtype], D, float(vv.abs().max()))
    return args, out, scale


KINDS = [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16"), ("e5m2", "bf16"), ("e5m2", "f16"),
         ("i8", "bf16"), ("i8", "f16"), ("u3", "bf16"), ("u3", "f16")]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind,dtype", KINDS)
def test_kinds(pkv, kind, dtype, D):
    """Whole prompts, chunks behind a longer context, and single tokens."""
    case(pkv, kind, dtype, new=[70, 1, 33, 200, 1], ctx=[70, 1, 160, 301, 500], D=D, seed=D)


@pytest.mark.parametrize("scales", ["block", "token"])
@pytest.mark.parametrize("kind,dtype", [k for k in KINDS if k[0] in R.QMAX])
def test_granular_scales(pkv, kind, dtype, scales):
    case(pkv, kind, dtype, new=[90, 1, 40], ctx=[90, 260, 300], scales=scales, seed=5)


@pytest.mark.parametrize("kind,D", [("bf16", 128), ("f16", 64), ("e4m3", 128), ("i8", 64)])
def test_xvec(pkv, kind, D):
    case(pkv, kind, "f16" if kind == "f16" else "bf16", new=[65, 3, 130], ctx=[65, 200, 130], layout="xvec", D=D, seed=6)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "u3"])
def test_dual_stacked_halves(pkv, kind):
    """K and V as strided halves of one buffer, head-major blocks."""
    case(pkv, kind, "bf16", new=[65, 3], ctx=[100, 200], dual=True, seed=7)


@pytest.mark.parametrize("BS", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_block_sizes(pkv, kind, BS):
    case(pkv, kind, "bf16", new=[50, 130, 7], ctx=[50, 333, 129], BS=BS, seed=BS)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 16, 17, 40, 64])
def test_groups(pkv, G):
    """Groups that do and do not divide a row tile."""
    case(pkv, "bf16", "bf16", new=[37, 1, 90], ctx=[37, 260, 290], H=1 if G > 16 else 3, G=G, seed=G)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257])
def test_lengths(pkv, n):
    """Prompt lengths around the tile edges, with and without a context
    before them, in one call."""
    case(pkv, "bf16", "bf16", new=[n, n, n], ctx=[n, n + 1, n + 128], seed=n)


def test_empty_sequences(pkv):
    """Sequences without new tokens between others, and contexts of zero."""
    case(pkv, "bf16", "bf16", new=[0, 5, 0, 0, 9, 0], ctx=[0, 5, 40, 0, 60, 0], seed=3)


def test_rows_that_see_nothing_are_zero(pkv):
    """More new tokens than cached ones: the first rows see no token."""
    ctx, new = [3, 0, 130, 1], [40, 5, 300, 2]
    args, out, scale = case(pkv, "bf16", "bf16", new=new, ctx=ctx, seed=4)
    at = 0
    for n, c in zip(new, ctx):
        assert (out[at:at + max(0, n - c)] == 0).all()
        at += n


@pytest.mark.parametrize("scale", [0.0, -0.11, 2.5, 1e-4])
def test_softmax_scales(pkv, scale):
    case(pkv, "bf16", "bf16", new=[130, 20], ctx=[130, 300], sm_scale=scale, seed=8)


@pytest.mark.parametrize("amp", [1e-3, 40.0])
@pytest.mark.parametrize("kind,dtype", [("f16", "f16"), ("e4m3", "f16"), ("u3", "f16"), ("bf16", "bf16")])
def test_value_ranges(pkv, kind, dtype, amp):
    """Small and large cache values, and with them small and large scales."""
    case(pkv, kind, dtype, new=[60, 2], ctx=[200, 300], amp=amp, scales="token" if kind == "e4m3" else "head",
         sm_scale=0.02, seed=9)


def test_many_short_sequences(pkv):
    g = torch.Generator().manual_seed(11)
    new = torch.randint(0, 4, (700,), generator=g).tolist()
    ctx = [n + int(torch.randint(0, 60, (1,), generator=g)) for n in new]
    case(pkv, "bf16", "bf16", new=new, ctx=ctx, H=1, G=2, seed=11)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "u3"])
def test_few_rows_long_context(pkv, kind):
    """Few rows over long contexts (spread over many SMs and joined)."""
    case(pkv, kind, "bf16", new=[1, 3], ctx=[9000, 5001], H=2, G=4, seed=12)


def test_long_prompt(pkv):
    case(pkv, "bf16", "bf16", new=[3001], ctx=[3001], H=1, G=4, seed=13)


def test_equal_to_decode(pkv):
    """One new token per sequence is a decode step."""
    ctx = [1, 17, 300, 1000]
    args, out, scale = case(pkv, "bf16", "bf16", new=[1] * 4, ctx=ctx, H=2, G=4, seed=14)
    q, cache, bt, st, cl = args
    dec = pkv.paged_decode(q, cache, bt, cl, sm_scale=scale)
    d = (dec.double() - out.double()).abs()
    # both within half a step of the weights' mean |v| (below 4 here) and of the output
    assert float(d.max()) <= 4 * R.half_step(torch.bfloat16) * 4


def test_strided_tensors(pkv):
    """q and out as slices of wider buffers, block tables and lengths with
    strides, rows behind the last sequence left as they were."""
    ctx, new, BS, H, G, D = [40, 150], [40, 70], 16, 2, 3, 128
    bt, P = R.tables(ctx, BS, seed=15)
    cache, kv, vv = R.make_cache(pkv, "bf16", P, BS, H, D, seed=15)
    g = torch.Generator().manual_seed(16)
    st = starts_of(new, first=4)
    T = st[-1] + 9
    wide = torch.randn((T, H * G + 2, D + 8), generator=g).to(torch.bfloat16).to(DEV)
    q = wide[:, 1:-1, :D]
    obuf = torch.full((T, 2 * H * G, D), 7.0, dtype=torch.bfloat16, device=DEV)
    out = obuf[:, ::2]
    btw = torch.stack([bt, bt], 2).to(DEV)[:, :, 0]
    meta = torch.full((2, 2), 99, dtype=torch.int32, device=DEV)
    meta[:, 0] = torch.tensor(ctx)
    sts = torch.tensor([[x, -1] for x in st], dtype=torch.int32, device=DEV)[:, 0]
    assert btw.stride(1) == 2 and meta[:, 0].stride(0) == 2 and sts.stride(0) == 2
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.paged_prefill(q, cache, btw, sts, meta[:, 0], out=out, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(out, R.prefill(q.cpu(), kv, vv, bt, st, ctx, D ** -0.5), torch.bfloat16, D, float(vv.abs().max()))
    assert (obuf[:, 1::2] == 7).all() and (out[:4] == 7).all() and (out[st[-1]:] == 7).all()


def test_unaligned_out(pkv):
    """An out whose rows are only 2-byte aligned."""
    ctx, new, BS, H, G, D = [40, 150], [40, 70], 16, 2, 4, 64
    bt, P = R.tables(ctx, BS, seed=17)
    cache, kv, vv = R.make_cache(pkv, "bf16", P, BS, H, D, seed=17)
    q = torch.randn((110, H * G, D), generator=torch.Generator().manual_seed(18)).to(torch.bfloat16).to(DEV)
    out = torch.empty((110, H * G, D + 1), dtype=torch.bfloat16, device=DEV)[..., 1:]
    st = starts_of(new)
    pkv.paged_prefill(q, cache, bt.to(DEV), torch.tensor(st, dtype=torch.int32, device=DEV),
                      torch.tensor(ctx, dtype=torch.int32, device=DEV), out=out)
    check(out, R.prefill(q.cpu(), kv, vv, bt, st, ctx, D ** -0.5), torch.bfloat16, D, float(vv.abs().max()))


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_poison_where_nothing_looks(pkv, kind, poison):
    """Every slot behind the contexts, and every block that no table names,
    holds NaN or infinities."""
    ctx, new, BS, H, G, D = [41, 150, 260], [41, 70, 2], 16, 2, 4, 128
    bt, P = R.tables(ctx, BS, seed=19)
    cache, kv, vv = R.make_cache(pkv, kind, P, BS, H, D, seed=19)
    seen = torch.zeros((P, BS), dtype=torch.bool)
    for b, c in enumerate(ctx):
        for t in range(c):
            seen[bt[b, t // BS], t % BS] = True
    for t in (cache.k_cache, cache.v_cache):
        t[~seen.to(DEV)] = poison
    q = torch.randn((113, H * G, D), generator=torch.Generator().manual_seed(20)).to(R.DT[kind])
    st = starts_of(new)
    out = pkv.paged_prefill(q.to(DEV), cache, bt.to(DEV), torch.tensor(st, dtype=torch.int32, device=DEV),
                            torch.tensor(ctx, dtype=torch.int32, device=DEV))
    check(out, R.prefill(q, kv, vv, bt, st, ctx, D ** -0.5), R.DT[kind], D, float(vv.abs().max()))


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_poison_in_the_future(pkv, what, poison):
    """A token whose row holds NaN or infinities: the rows before it do not
    see it; those that see it are not finite."""
    n, at, BS, H, G, D = 200, 137, 16, 2, 4, 128
    bt, P = R.tables([n], BS, seed=21)
    cache, kv, vv = R.make_cache(pkv, "bf16", P, BS, H, D, seed=21)
    buf = cache.k_cache if what == "k" else cache.v_cache
    buf[int(bt[0, at // BS]), at % BS] = poison
    q = torch.randn((n, H * G, D), generator=torch.Generator().manual_seed(22)).abs().to(torch.bfloat16)
    out = pkv.paged_prefill(q.to(DEV), cache, bt.to(DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV),
                            torch.tensor([n], dtype=torch.int32, device=DEV))
    ref = R.prefill(q, kv, vv, bt, [0, n], [n], D ** -0.5)
    cut = tuple(r[:at] for r in ref)
    check(out[:at], cut, torch.bfloat16, D, float(vv.abs().max()))
    assert not torch.isfinite(out[at:]).any()


def test_bad_data_is_flagged(pkv):
    """Bad block ids are left out, lengths outside the table are clamped,
    q_starts that decrease leave their sequence out; the other sequences'
    rows stay right."""
    ctx, new, BS, H, G, D = [100, 60, 90], [30, 60, 20], 16, 2, 4, 128
    bt, P = R.tables(ctx, BS, seed=23)
    cache, kv, vv = R.make_cache(pkv, "bf16", P, BS, H, D, seed=23)
    q = torch.randn((110, H * G, D), generator=torch.Generator().manual_seed(24)).to(torch.bfloat16)
    st = starts_of(new)
    ref = R.prefill(q, kv, vv, bt, st, ctx, D ** -0.5)
    vmax = float(vv.abs().max())

    def run(bt_, st_, ctx_):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = torch.full((110, H * G, D), 5.0, dtype=torch.bfloat16, device=DEV)
        pkv.paged_prefill(q.to(DEV), cache, bt_.to(DEV), torch.tensor(st_, dtype=torch.int32, device=DEV),
                          torch.tensor(ctx_, dtype=torch.int32, device=DEV), out=out, err_flag=err)
        torch.cuda.synchronize()
        return out, int(err.item())

    for wrong in (-1, P, 2 ** 31 - 1):
        b2 = bt.clone()
        b2[1, 2] = wrong
        out, e = run(b2, st, ctx)
        assert e == pkv.pkv.DEVERR_BLOCK_RANGE
        check(out[:30], tuple(r[:30] for r in ref), torch.bfloat16, D, vmax)
        check(out[90:], tuple(r[90:] for r in ref), torch.bfloat16, D, vmax)
        # rows of sequence 1 before the bad block are right, and later ones
        # are attention over the other blocks' tokens
        check(out[30:62], tuple(r[30:62] for r in ref), torch.bfloat16, D, vmax)
        left = torch.cat([torch.arange(32), torch.arange(48, 60)])
        ids = bt[1].long()[left // BS]
        k, v = kv[ids, left % BS], vv[ids, left % BS]
        s = torch.einsum("hgd,chd->hgc", q[89].double().view(H, G, D), k) * D ** -0.5
        want = torch.einsum("hgc,chd->hgd", torch.softmax(s, -1), v).reshape(H * G, D)
        assert float((out[89].double().cpu() - want).abs().max()) < 0.03
    out, e = run(bt, st, [100, -5, 90])
    assert e == pkv.pkv.DEVERR_CONTEXT_RANGE and (out[30:90] == 0).all()
    check(out[:30], tuple(r[:30] for r in ref), torch.bfloat16, D, vmax)
    out, e = run(bt, st, [7 * BS + 1, 60, 90])
    assert e & pkv.pkv.DEVERR_CONTEXT_RANGE
    check(out[30:], tuple(r[30:] for r in ref), torch.bfloat16, D, vmax)
    # sequence 1 would own rows 30 .. -1 and 2 rows 0 .. 109 of other sequences: only 1 is out of order
    out, e = run(bt, [0, 30, 20, 110], ctx)
    assert e == pkv.pkv.DEVERR_QSTART_RANGE
    out, e = run(bt, [0, 30, 90, 400], ctx)
    assert e == pkv.pkv.DEVERR_QSTART_RANGE
    check(out[:90], tuple(r[:90] for r in ref), torch.bfloat16, D, vmax)
    assert (out[90:] == 5).all()


def test_graph_replay_with_new_lengths(pkv):
    """A captured call replays with other lengths, starts and tables."""
    BS, H, G, D = 16, 2, 4, 128
    runs = [([100, 60], [100, 60]), ([3, 150], [300, 170]), ([0, 1], [0, 310])]
    T, P = 160, 64
    cache, kv, vv = R.make_cache(pkv, "bf16", P, BS, H, D, seed=25)
    q = torch.randn((T, H * G, D), generator=torch.Generator().manual_seed(26)).to(torch.bfloat16).to(DEV)
    bt = torch.zeros((2, 20), dtype=torch.int32, device=DEV)
    st = torch.zeros(3, dtype=torch.int32, device=DEV)
    cl = torch.zeros(2, dtype=torch.int32, device=DEV)
    out = torch.zeros_like(q)
    ws = torch.empty(pkv.prefill_workspace_bytes(q, cache, bt), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    pkv.paged_prefill(q, cache, bt, st, cl, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkv.paged_prefill(q, cache, bt, st, cl, out=out, workspace=ws)
    for i, (new, ctx) in enumerate(runs):
        t, _ = R.tables(ctx, BS, extra=P - sum(-(-c // BS) for c in ctx), seed=i, width=20)
        s = starts_of(new)
        bt.copy_(t)
        st.copy_(torch.tensor(s))
        cl.copy_(torch.tensor(ctx))
        ws.fill_(255)                    # NaN everywhere: the workspace needs no initialisation
        for _ in range(2):
            out.fill_(3.0)
            graph.replay()
            torch.cuda.synchronize()
            check(out, R.prefill(q.cpu(), kv, vv, t, s, ctx, D ** -0.5), torch.bfloat16, D, float(vv.abs().max()))
            assert (out[s[-1]:] == 3).all()


def test_repeated_calls_are_bit_identical(pkv):
    args, out, scale = case(pkv, "bf16", "bf16", new=[300, 1, 40], ctx=[300, 3000, 1000], H=2, G=4, seed=27)
    for _ in range(3):
        assert torch.equal(pkv.paged_prefill(*args, sm_scale=scale), out)


def test_other_stream(pkv):
    """A call on a stream of its own, its buffers allocated by the call."""
    args, out, scale = case(pkv, "bf16", "bf16", new=[300, 40], ctx=[300, 1000], H=2, G=4, seed=28)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [pkv.paged_prefill(*args, sm_scale=scale, stream=s) for _ in range(4)]
    s.synchronize()
    for o in got:
        assert torch.equal(o, out)


def test_thousands_of_sequences(pkv):
    """More sequences than the kernel counts one by one."""
    g = torch.Generator().manual_seed(31)
    new = torch.randint(0, 3, (2500,), generator=g).tolist()
    ctx = [n + int(torch.randint(0, 20, (1,), generator=g)) for n in new]
    case(pkv, "bf16", "bf16", new=new, ctx=ctx, H=1, G=1, D=64, BS=8, seed=31)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_row_tiles_of_every_size(pkv, kind):
    """Runs of row tiles with one and two subtiles and key tiles odd and even
    in number, many per CTA, in one call and again."""
    new = [129, 1, 260, 33, 64, 1, 300, 140, 5, 513, 100, 31] * 6
    g = torch.Generator().manual_seed(32)
    ctx = [n + int(torch.randint(0, 700, (1,), generator=g)) for n in new]
    args, out, scale = case(pkv, kind, "bf16", new=new, ctx=ctx, H=2, G=2, seed=32)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for _ in range(20):
        assert torch.equal(pkv.paged_prefill(*args, sm_scale=scale, err_flag=err), out)
    assert int(err.item()) == 0


def test_two_streams_at_once(pkv):
    """Calls on two streams, each with a workspace of its own."""
    a, out_a, scale = case(pkv, "bf16", "bf16", new=[300, 40], ctx=[300, 1000], H=2, G=4, seed=33)
    b, out_b, _ = case(pkv, "e4m3", "bf16", new=[200, 7], ctx=[900, 1000], H=2, G=4, seed=34)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(pkv.paged_prefill(*a, sm_scale=scale, stream=s), pkv.paged_prefill(*b, sm_scale=scale, stream=t))
           for _ in range(8)]
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, out_a) and torch.equal(y, out_b)


@pytest.mark.parametrize("D", [64, 128])
def test_packed_rows_off_the_word(pkv, D):
    """3-bit rows at odd byte strides (no tensor map, no 4-byte loads)."""
    BS, H, G, ctx, new = 16, 2, 3, [70, 200], [70, 9]
    bt, P = R.tables(ctx, BS, seed=35)
    cache, kv, vv = R.make_cache(pkv, "u3", P, BS, H, D, seed=35)
    row = 3 * D // 8
    halves = []
    for t in (cache.k_cache, cache.v_cache):
        wide = torch.zeros((P, (BS * H * (row + 1) + 15) // 16 * 16), dtype=torch.uint8, device=DEV)
        view = wide.as_strided((P, BS, H, row), (wide.stride(0), H * (row + 1), row + 1, 1))
        view.copy_(t)
        halves.append(view)
    odd = pkv.KVCache("u3", *halves, k_qscale=cache.k_qscale, k_qzero=cache.k_qzero, v_qscale=cache.v_qscale,
                      v_qzero=cache.v_qzero)
    q = torch.randn((79, H * G, D), generator=torch.Generator().manual_seed(36)).bfloat16()
    st = starts_of(new)
    dev = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (st, ctx)]
    out = pkv.paged_prefill(q.to(DEV), odd, bt.to(DEV), *dev)
    check(out, R.prefill(q, kv, vv, bt, st, ctx, D ** -0.5), torch.bfloat16, D, float(vv.abs().max()))
    slots = torch.arange(P * BS, device=DEV)
    for x, y in zip(pkv.kv_gather(odd, slots), pkv.kv_gather(cache, slots)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pad", [4, 8, 16])
def test_packed_rows_apart(pkv, pad, D):
    """3-bit rows in wider slots; each CTA takes more key tiles than are in flight."""
    BS, H, G, ctx, new = 16, 4, 8, [2300, 1100], [1300, 3]
    bt, P = R.tables(ctx, BS, seed=38)
    cache, kv, vv = R.make_cache(pkv, "u3", P, BS, H, D, seed=38)
    row = 3 * D // 8 + pad
    halves = []
    for t in (cache.k_cache, cache.v_cache):
        view = torch.full((P, BS, H, row), 255, dtype=torch.uint8, device=DEV)[..., :3 * D // 8]
        view.copy_(t)
        halves.append(view)
    apart = pkv.KVCache("u3", *halves, k_qscale=cache.k_qscale, k_qzero=cache.k_qzero, v_qscale=cache.v_qscale,
                        v_qzero=cache.v_qzero)
    q = torch.randn((1303, H * G, D), generator=torch.Generator().manual_seed(39)).bfloat16()
    st = starts_of(new)
    dev = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (st, ctx)]
    out = pkv.paged_prefill(q.to(DEV), apart, bt.to(DEV), *dev)
    check(out, R.prefill(q, kv, vv, bt, st, ctx, D ** -0.5), torch.bfloat16, D, float(vv.abs().max()))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("BS", [8, 64])
def test_xvec_long(pkv, kind, D, BS):
    """X-vectorised caches; each CTA takes more key tiles than are in flight,
    in row tiles of one subtile and of two."""
    case(pkv, kind, "f16" if kind == "f16" else "bf16", new=[1300, 5, 1, 140], ctx=[2300, 2003, 1, 900], H=4, G=8,
         layout="xvec", D=D, BS=BS, seed=40)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind,scales", [("bf16", "head"), ("e4m3", "token"), ("e5m2", "block"), ("i8", "head"),
                                         ("i8", "token"), ("u3", "head")])
def test_long_shares(pkv, kind, scales, D):
    """Row-major caches, likewise."""
    case(pkv, kind, "bf16", new=[1300, 5, 1, 140], ctx=[2300, 2003, 1, 900], H=4, G=8, scales=scales, D=D, seed=41)


def test_no_blocks_and_no_table(pkv):
    """An empty pool, or a block table without columns: nothing to see."""
    q = torch.randn((5, 4, 64), generator=torch.Generator().manual_seed(37)).half().to(DEV)
    st = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    k = torch.zeros((0, 16, 2, 64), dtype=torch.float16, device=DEV)
    for cache, cols, ctx, flag in ((pkv.KVCache("f16", k, k), 2, 20, pkv.pkv.DEVERR_BLOCK_RANGE),
                                   (pkv.KVCache.allocate("f16", 3, 16, 2, 64, fill=255), 0, 0, 0),
                                   (pkv.KVCache.allocate("f16", 3, 16, 2, 64, fill=255), 0, 7, pkv.pkv.DEVERR_CONTEXT_RANGE)):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = pkv.paged_prefill(q, cache, torch.zeros((1, cols), dtype=torch.int32, device=DEV), st,
                                torch.tensor([ctx], dtype=torch.int32, device=DEV), err_flag=err)
        assert int(err.item()) == flag and (out == 0).all()


def test_far_blocks(pkv):
    """Blocks beyond 2^32 bytes into the pool."""
    BS, H, D, G = 16, 8, 128, 1
    P = (1 << 32) // (BS * H * D * 2) + 64
    new, ctx = [40, 1], [100, 150]
    bt, near = R.tables(ctx, BS, seed=29)
    small, kv, vv = R.make_cache(pkv, "bf16", near, BS, H, D, seed=29)
    k = torch.empty((P, BS, H, D), dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    k[-near:] = small.k_cache
    v[-near:] = small.v_cache
    q = torch.randn((41, H * G, D), generator=torch.Generator().manual_seed(30)).to(torch.bfloat16)
    st = starts_of(new)
    far = torch.where(bt >= 0, bt + P - near, bt)
    dev = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (st, ctx)]
    out = pkv.paged_prefill(q.to(DEV), pkv.KVCache("bf16", k, v), far.to(DEV), *dev)
    assert torch.equal(out, pkv.paged_prefill(q.to(DEV), small, bt.to(DEV), *dev))
    check(out, R.prefill(q, kv, vv, bt, st, ctx, D ** -0.5), torch.bfloat16, D, float(vv.abs().max()))
