"""Block tables, rows and slots from request lengths, and blocks given back,
against a host's loops: every number equal."""
import random

import pytest
import torch

import paged_kv_cache_num_gb300 as pkv
from paged_kv_cache_num_gb300 import pkv as P_

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def ceil(a, b):
    return -(-a // b)


def extend(table, cached, new, stack, count, BS, N, cap):
    """The definition, request by request.  Returns the outputs and the error bits."""
    err, used, rows = 0, 0, []
    if not 0 <= count <= len(stack):
        err |= P_.DEVERR_POOL_RANGE
        count = min(max(count, 0), len(stack))
    table = [r[:] for r in table]
    starts, lens, full = [0], [], False
    for b, (a, n) in enumerate(zip(cached, new)):
        if not 0 <= a <= cap:
            err |= P_.DEVERR_CONTEXT_RANGE
            a = min(max(a, 0), cap)
        if n < 0 or a + n > cap:
            err |= P_.DEVERR_CONTEXT_RANGE
            n = 0
        have, need = ceil(a, BS), ceil(a + n, BS) - ceil(a, BS)
        if full or len(rows) + n > N or used + need > count:
            full = True
            if n > 0:
                err |= P_.DEVERR_POOL_RANGE
            n = need = 0
        for j in range(need):
            table[b][have + j] = stack[count - 1 - used - j]
        used += need
        rows += [(b, a + i, table[b][(a + i) // BS] * BS + (a + i) % BS) for i in range(n)]
        starts.append(len(rows))
        lens.append(a + n)
    rows += [(-1, -1, -1)] * (N - len(rows))
    return table, lens, starts, [list(c) for c in zip(*rows)] if rows else [[], [], []], count - used, err


def trim(table, ctx, keep, stack, count, BS, cap):
    err = 0
    if not 0 <= count <= len(stack):
        err |= P_.DEVERR_POOL_RANGE
        count = min(max(count, 0), len(stack))
    stack, out, full = stack[:], [], False
    for b, (t, k) in enumerate(zip(ctx, keep)):
        if not 0 <= t <= cap:
            err |= P_.DEVERR_CONTEXT_RANGE
            t = min(max(t, 0), cap)
        k = min(max(k, 0), t)
        drop = range(ceil(k, BS), ceil(t, BS))
        if full or count + len(drop) > len(stack):
            full = True
            err |= P_.DEVERR_POOL_RANGE if len(drop) or k else 0
            out.append(t)
            continue
        for j in drop:
            stack[count] = table[b][j]
            count += 1
        out.append(k)
    return out, stack, count, err


def state(B, BS, M, seed, most=None):
    """Random lengths, a table with their blocks and a stack with the rest."""
    r = random.Random(seed)
    cached = [r.randint(0, most if most is not None else M * BS) for _ in range(B)]
    ids = list(range(sum(ceil(a, BS) for a in cached) + r.randint(0, 3 * B + 5)))
    r.shuffle(ids)
    table = [[-9] * M for _ in range(B)]
    for b, a in enumerate(cached):
        for j in range(ceil(a, BS)):
            table[b][j] = ids.pop()
    return r, cached, table, ids + [-5] * r.randint(0, 4), len(ids)


def run_extend(table, cached, new, stack, count, BS, N, **kw):
    bt, fb = i32(table).view(len(cached), -1), i32(stack)
    err = i32([0])
    ctx, starts, req, pos, slots, left = pkv.extend_tables(bt, i32(cached), i32(new), fb, i32([count]), BS, N, err_flag=err, **kw)
    assert fb.tolist() == stack
    return bt.tolist(), ctx.tolist(), starts.tolist(), [req.tolist(), pos.tolist(), slots.tolist()], left.item(), err.item()


@pytest.mark.parametrize("B,BS,M,new,N", [(1, 16, 4, 1, 1), (1, 1, 9, 9, 16), (3, 16, 8, 20, 64), (33, 8, 20, 40, 1500), (64, 32, 10, 1, 256), (700, 16, 12, 9, 4000),
                                          (513, 64, 6, 200, 60000), (5000, 4, 9, 3, 9000), (16384, 16, 2, 2, 20000), (2, 16, 4000, 50000, 90000)])
@pytest.mark.parametrize("seed", [1, 2])
def test_extend(B, BS, M, new, N, seed):
    """Requests without new tokens among them; more often than not the pool or the
    rows run out in the middle."""
    r, cached, table, stack, count = state(B, BS, M, 10 * B + seed, most=M * BS // 2)
    more = [r.choice([0, 1, r.randint(0, new)]) for _ in range(B)]
    want = extend(table, cached, more, stack, count, BS, N, M * BS)
    assert run_extend(table, cached, more, stack, count, BS, N) == want


def test_extend_no_requests_and_no_rows():
    bt = torch.zeros((0, 5), dtype=torch.int32, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    ctx, starts, req, pos, slots, left = pkv.extend_tables(bt, none, none, i32([1, 2]), i32([2]), 16, 5)
    assert starts.tolist() == [0] and left.item() == 2 and ctx.numel() == 0
    assert req.tolist() == pos.tolist() == slots.tolist() == [-1] * 5
    assert run_extend([[3, 4]], [20], [0], [], 0, 16, 0) == ([[3, 4]], [20], [0, 0], [[], [], []], 0, 0)
    # no room for a row: flagged
    assert run_extend([[3, 4]], [20], [1], [7], 1, 16, 0)[1:] == ([20], [0, 0], [[], [], []], 1, P_.DEVERR_POOL_RANGE)


@pytest.mark.parametrize("cached,new", [([-1, 5], [2, 2]), ([65, 5], [0, 2]), ([64, 5], [1, 2]), ([0, 5], [-3, 2]), ([0, 5], [2 ** 31 - 1, 2]), ([-2 ** 31, 64], [64, 0]),
                                        ([2 ** 31 - 1, 64], [2 ** 31 - 1, -2 ** 31])])
def test_extend_bad_lengths(cached, new):
    table, stack = [[10, 11, 12, 13], [20, 21, 22, 23]], [1, 2, 3, 4, 5]
    assert run_extend(table, cached, new, stack, 5, 16, 70) == extend(table, cached, new, stack, 5, 16, 70, 64)


@pytest.mark.parametrize("count", [-1, 6, 2 ** 31 - 1, -2 ** 31])
def test_extend_bad_counts(count):
    table, stack = [[10, 11, 12, 13], [20, 21, 22, 23]], [1, 2, 3, 4, 5]
    assert run_extend(table, [5, 6], [20, 20], stack, count, 16, 70) == extend(table, [5, 6], [20, 20], stack, count, 16, 70, 64)


def test_extend_in_place_strided_and_captured():
    """Lengths and count onto themselves, strided tables, the same graph step after step."""
    B, BS, M, N = 9, 4, 30, 16
    r, cached, table, stack, count = state(B, BS, M, 3, most=40)
    stack = stack[:count] + list(range(10000, 10060))
    count = len(stack)
    wide = torch.full((B, 2 * M), -4, dtype=torch.int32, device=DEV)
    bt = wide[:, ::2]
    bt.copy_(i32(table))
    lens = i32([[c, 0] for c in cached])[:, 0]
    new, fb, left = i32([1] * B), i32(stack), i32([count])
    out = [torch.empty(n, dtype=d, device=DEV) for n, d in ((B + 1, torch.int32), (N, torch.int32), (N, torch.int32), (N, torch.int64))]
    step = lambda: pkv.extend_tables(bt, lens, new, fb, left, BS, context_lens=lens, q_starts=out[0], req=out[1], pos=out[2], slot_mapping=out[3], free_left=left)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.synchronize()
    for i in range(12):
        n = [r.randint(0, 2) for _ in range(B)]
        while sum(n) > N:
            n[r.randrange(B)] = 0
        new.copy_(i32(n))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        table, cached, starts, rows, count, err = extend(table, cached, n, stack, count, BS, N, M * BS)
        assert err == 0
        assert bt.tolist() == table and lens.tolist() == cached and left.item() == count
        assert out[0].tolist() == starts and [o.tolist() for o in out[1:]] == rows
    assert (wide[:, 1::2] == -4).all()


def run_trim(table, ctx, keep, stack, count, BS, **kw):
    bt, fb, err = i32(table).view(len(ctx), -1), i32(stack), i32([0])
    kept, left = pkv.trim_tables(bt, i32(ctx), i32(keep), fb, i32([count]), BS, err_flag=err, **kw)
    assert bt.tolist() == table
    return kept.tolist(), fb.tolist(), left.item(), err.item()


@pytest.mark.parametrize("B,BS,M", [(1, 16, 4), (1, 1, 3000), (3, 16, 8), (64, 16, 40), (700, 8, 30), (5000, 4, 9), (16384, 16, 2)])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_trim(B, BS, M, seed):
    r, ctx, table, stack, count = state(B, BS, M, B + seed)
    keep = [r.choice([0, t, r.randint(0, t), t + 5, -2, 2 ** 31 - 1, max(0, t - 1)]) for t in ctx]
    if seed < 3:                                                     # else the stack is too small
        stack = stack + [-5] * sum(ceil(t, BS) for t in ctx)
    assert run_trim(table, ctx, keep, stack, count, BS) == trim(table, ctx, keep, stack, count, BS, M * BS)


def test_trim_bad_values():
    table, stack = [[10, 11, 12, 13], [20, 21, 22, 23]], [1, 2, 3, 4, 5, 0, 0, 0, 0, 0, 0, 0, 0]
    for ctx, keep, count in (([-4, 70], [3, 3], 5), ([64, 17], [0, 0], -1), ([64, 17], [0, 0], 14), ([33, 17], [16, 1], 12)):
        assert run_trim(table, ctx, keep, stack, count, 16) == trim(table, ctx, keep, stack, count, 16, 64)


def test_trim_undoes_extend():
    """Blocks that were handed out and given back are those of before."""
    B, BS, M = 40, 8, 30
    r, cached, table, stack, count = state(B, BS, M, 5, most=60)
    stack = stack[:count] + list(range(1000, 1300))
    count = len(stack)
    bt, fb, left = i32(table), i32(stack), i32([count])
    lens = i32(cached)
    new = i32([r.randint(0, 40) for _ in range(B)])
    ctx = pkv.extend_tables(bt, lens, new, fb, left, BS, 2000, free_left=left)[0]
    assert torch.equal(ctx, lens + new)
    kept, _ = pkv.trim_tables(bt, ctx, lens, fb, left, BS, kept_lens=ctx, free_left=left)
    assert kept is ctx and torch.equal(kept, lens) and left.item() == count
    assert sorted(fb.tolist()) == sorted(stack)
    assert pkv.trim_tables(bt, lens, i32([0] * B), i32(stack + [0] * 400), left, BS)[1].item() == count + sum(ceil(a, BS) for a in cached)


@pytest.mark.parametrize("kind", ["u4", "bf16"])
def test_a_serving_loop(kind):
    """Prompts and decode steps of requests that come and go: tables from lengths,
    norm and rotation in the append's pass, attention over what is cached --
    against attention over the same rows kept one after another."""
    from tests import prompt_refs as R
    from tests import u4_refs as U
    BS, H, G, D, P, B, M = 16, 2, 4, 128, 60, 4, 20
    r = random.Random(8)
    cache = pkv.KVCache.allocate(kind, P, BS, H, D, fill=0)
    bt = torch.zeros((B, M), dtype=torch.int32, device=DEV)
    fb, left, lens = torch.randperm(P, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(DEV), i32([P]), i32([0] * B)
    half = D // 2
    ang = torch.arange(400, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    cs = torch.cat([ang.cos(), ang.sin()], -1).float().to(DEV)
    w = (1 + 0.2 * torch.randn(D, generator=torch.Generator().manual_seed(2))).to(DEV)
    err = i32([0])
    kept = [torch.zeros((0, H, D), dtype=torch.float64) for _ in range(2 * B)]       # dequantised K and V of each request
    tops = [t.clone() for t in kept]
    ctx = [0] * B
    for step in range(9):
        new = [r.randint(20, 60) if c == 0 else 1 for c in ctx]
        N = ceil(sum(new), 32) * 32
        lens, starts, req, pos, slots, left = pkv.extend_tables(bt, lens, i32(new), fb, left, BS, N, err_flag=err)
        g = torch.Generator().manual_seed(100 + step)
        qkv = torch.randn((N, H * G + 2 * H, D), generator=g).bfloat16().to(DEV)
        q, k, v = qkv.split([H * G, H, H], 1)
        qr = pkv.norm_rope_append(q, k, v, cs, pos, slots, cache, w, w, err_flag=err)
        _, kr = pkv.norm_rope(q, k, cs, pos, w, w)
        live = sum(new)
        out = pkv.paged_prefill(qr, cache, bt, starts, lens, err_flag=err)
        if max(new) == 1:
            dec = pkv.paged_decode(qr[:live], cache, bt, lens, err_flag=err)
        ctx = [c + n for c, n in zip(ctx, new)]
        assert lens.tolist() == ctx
        at = 0
        for b, n in enumerate(new):
            for half_, x in ((0, kr), (1, v)):
                rows = x[at:at + n].cpu()
                if kind == "u4":
                    c, s, z = U.quantise(rows)
                    val = (c.double() - z.double()[..., None]) * s.double()[..., None]
                    top = (c.double() + z.double()[..., None]) * s.double()[..., None]
                else:
                    val = rows.double()
                    top = val.abs()
                kept[2 * b + half_] = torch.cat([kept[2 * b + half_], val])
                tops[2 * b + half_] = torch.cat([tops[2 * b + half_], top])
            at += n
        # a plain pool: request b's rows in block b, as long as the longest
        L = max(ctx)
        pad = lambda x: torch.cat([x, x.new_zeros((L - x.shape[0], H, D))])  # noqa: E731
        vals = [torch.stack([pad(kept[2 * b + i]) for b in range(B)]) for i in (0, 1)]
        top = [torch.stack([pad(tops[2 * b + i]) for b in range(B)]) for i in (0, 1)]
        st = starts.tolist()
        plain = torch.arange(B, dtype=torch.int32)[:, None]
        parts = U.prefill_parts(qr[:live].cpu(), vals, top, plain, st, ctx, D ** -0.5)
        if kind == "u4":
            close = lambda x: U.close(x, parts, 8.0, torch.bfloat16, D)  # noqa: E731
        else:
            ref = R.prefill(qr[:live].cpu(), vals[0], vals[1], plain, st, ctx, D ** -0.5)

            def close(x):
                err_ = (x.double().cpu() - ref[0]).abs()
                assert (err_ <= R.prefill_tolerance(*ref, 8.0, torch.bfloat16, D)).all()
        close(out[:live])
        if max(new) == 1:
            close(dec)
        if step % 4 == 3:                                            # a request ends, another loses its last tokens
            keep = ctx[:]
            keep[step % B], keep[(step + 1) % B] = 0, ctx[(step + 1) % B] - 3
            lens, left = pkv.trim_tables(bt, lens, i32(keep), fb, left, BS, err_flag=err)
            ctx = keep
            for b in range(B):
                for i in (0, 1):
                    kept[2 * b + i], tops[2 * b + i] = kept[2 * b + i][:ctx[b]], tops[2 * b + i][:ctx[b]]
        assert left.item() == P - sum(ceil(c, BS) for c in ctx)
    assert err.item() == 0
