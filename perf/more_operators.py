"""Cases of the operators around a 4-bit cache and of a serving step's
beginning: attention over a cache held in 4 bits (paged_decode and
paged_prefill of a "u4" cache), rows put into it and read back (kv_append,
kv_gather), the norm and rotation of queries and keys in the pass that appends
them (norm_rope_append), and block tables, slots and row numbers made from
request lengths (extend_tables, trim_tables).

A case is a dict of plain values; prepare() makes the inputs on the GPU from
a seed, run() makes one pass (the plain form in elementary torch operations,
or the library's calls where `own` is set), exact() gives the result in 64
bits, work() what a pass has to move and compute.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6                           # of the norms
FAR = 40960                          # positions of the rotation's table


# ---------------------------------------------------------------- cases
def listed():
    att = {"dtype": "bf16", "dim": 128, "block": 16}
    dec, pre = dict(att, op="decode"), dict(att, op="prefill")
    app = {"op": "append", "dtype": "bf16", "dim": 128, "block": 16, "kv_heads": 8}
    rot = {"op": "rope", "dtype": "bf16", "dim": 128, "block": 16, "heads": 32, "kv_heads": 8}
    tab = {"op": "tables", "block": 16}
    return [
        # one chat turn's next token: a single sequence, where latency counts
        dict(dec, name="decode_one", heads=32, kv_heads=8, batch=1, ctx_lo=700, ctx_hi=700, mix=1),
        # a decode step over long contexts with grouped heads, the shape that 8-bit caches are used for
        dict(dec, name="decode_long", heads=64, kv_heads=8, block=32, batch=16, ctx_lo=16384, ctx_hi=32768, mix=2),
        # a decode step of a multi-head model, whose cache is the largest per token
        dict(dec, name="decode_mha", dtype="f16", heads=32, kv_heads=32, batch=32, ctx_lo=1024, ctx_hi=8192, mix=3),
        # many short requests of a small model with an odd group, in larger blocks
        dict(dec, name="decode_small_heads", heads=40, kv_heads=8, dim=64, block=64, batch=48, ctx_lo=1, ctx_hi=5000, mix=4),
        # chunked prompts over long contexts
        dict(pre, name="prefill_chunks", heads=64, kv_heads=8, block=32, batch=4, new_lo=400, new_hi=512, ctx_lo=8192, ctx_hi=16384, mix=5),
        # a few drafted tokens per sequence checked against the cache
        dict(pre, name="prefill_draft", dtype="f16", heads=32, kv_heads=8, batch=24, new_lo=1, new_hi=8, ctx_lo=500, ctx_hi=4000, mix=6),
        # one decode step's rows, stored and looked at again
        dict(app, name="append_step", tokens=64),
        # a batch of prompts stored, then read back to move them elsewhere
        dict(app, name="append_prompt", dtype="f16", tokens=40001),
        # one decode step: norms, rotation and append of a token per sequence
        dict(rot, name="rope_step", rot=128, pairs=False, norm=True, tokens=64),
        # prompts of a model with partly rotated heads, in the layout that the projection leaves
        dict(rot, name="rope_prompt", rot=64, pairs=True, norm=True, tokens=20011),
        # a decode step with drafted tokens: blocks handed out, then those of rejected tokens taken back
        dict(tab, name="tables_draft", batch=64, len_hi=4096, new_lo=1, new_hi=8, trim=True, mix=7),
        # many prompts scheduled at once
        dict(tab, name="tables_prompt", batch=601, len_hi=2000, new_lo=0, new_hi=500, trim=False, mix=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "append", "rope", "tables"])
    block = rng.choice([16, 16, 32, 64])
    if op == "tables":
        batch = _log_int(rng, 1, 2000)
        new_hi = _log_int(rng, 1, max(2, 150000 // batch))
        return {"op": op, "block": block, "batch": batch, "len_hi": _log_int(rng, 1, 6000), "new_lo": rng.randint(0, new_hi), "new_hi": new_hi,
                "trim": rng.choice([True, False]), "mix": rng.randint(1, 10 ** 6)}
    case = {"op": op, "dtype": rng.choice(["bf16", "f16"]), "dim": rng.choice([64, 128, 128]), "block": block}
    if op == "append":
        heads = rng.randint(1, 24)
        return case | {"kv_heads": heads, "tokens": _log_int(rng, 1, 320000 // heads)}
    if op == "rope":
        kv, group = rng.randint(1, 10), rng.randint(1, 8)
        rot = rng.choice([case["dim"], case["dim"], case["dim"] // 2, 32])
        return case | {"heads": kv * group, "kv_heads": kv, "rot": rot, "pairs": rng.choice([True, False]), "norm": rng.choice([True, True, False]),
                       "tokens": _log_int(rng, 1, 480000 // (kv * (group + 2)))}
    kv, group = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    case |= {"kv_heads": kv, "heads": kv * group, "mix": rng.randint(1, 10 ** 6)}
    if op == "decode":
        batch = _log_int(rng, 1, 128)
        ctx_hi = _log_int(rng, 1, min(32768, max(2, 3000000 // (batch * kv))))
        return case | {"batch": batch, "ctx_lo": rng.randint(1, ctx_hi), "ctx_hi": ctx_hi}
    batch = _log_int(rng, 1, 32)
    new_hi = _log_int(rng, 1, max(2, 3000 // batch))
    new_lo = rng.randint(1, new_hi)
    ctx_hi = rng.choice([0, _log_int(rng, new_hi, 8192)])
    # no more query-key pairs than the chunked prompts'
    while batch * kv * group * new_hi * max(new_hi, ctx_hi) > 1.0e9:
        batch, new_hi = max(1, batch // 2), max(1, new_hi * 3 // 4)
        new_lo = min(new_lo, new_hi)
    return case | {"batch": batch, "new_lo": new_lo, "new_hi": new_hi, "ctx_lo": ctx_hi // 4, "ctx_hi": ctx_hi}


def _lengths(c):
    """(new tokens, context length) of each sequence of a decode or prefill case."""
    r = random.Random(c["mix"])
    new = [r.randint(c.get("new_lo", 1), c.get("new_hi", 1)) for _ in range(c["batch"])]
    return new, [max(n, r.randint(c["ctx_lo"], c["ctx_hi"])) for n in new]


def _requests(c):
    """(cached, new, kept) tokens of each request of a tables case."""
    r = random.Random(c["mix"])
    cached = [r.randint(0, c["len_hi"]) for _ in range(c["batch"])]
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["batch"])]
    # a drafted token is kept or not; one request in eight ends and gives everything back
    kept = [0 if r.random() < 0.125 else a + r.randint(0, n) for a, n in zip(cached, new)]
    return cached, new, kept


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _pack4(codes):
    """[..., D] codes of 4 bits -> [..., D / 2] bytes, the even element in the low half."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _head_major(P, BS, H, dtype):
    """[P, BS, H] seen through storage [P, H, BS], as the library allocates scales and zeros."""
    return torch.zeros((P, H, BS), dtype=dtype, device=DEV).transpose(1, 2)


def _row_codes(x):
    """Rows [..., D] in 32 bits -> (codes, scale, zero): the range of a row and zero in 15 steps."""
    lo, hi = x.amin(-1, keepdim=True).clamp(max=0.0), x.amax(-1, keepdim=True).clamp(min=0.0)
    # divided by a tensor: by a Python number it would be a product with the reciprocal
    scale = ((hi - lo) / torch.full((), 15.0, device=x.device)).clamp(max=65504.0).to(torch.float16)
    s = scale.float()
    some = s > 0
    s = torch.where(some, s, torch.ones_like(s))
    zero = torch.where(some, (-lo / s).round().clamp(0, 15), torch.zeros_like(s))
    codes = torch.where(some, ((x / s).round() + zero).clamp(0, 15), torch.zeros_like(x))
    return codes.to(torch.uint8), scale[..., 0], zero[..., 0].to(torch.uint8)


def _half_cache(c, P, g):
    """One of K and V: packed rows, their scales and zeros."""
    BS, H, D = c["block"], c["kv_heads"], c["dim"]
    codes, scale, zero = _row_codes(_randn((P, BS, H, D), g))
    s = {"data": _pack4(codes), "scale": _head_major(P, BS, H, torch.float16), "zero": _head_major(P, BS, H, torch.uint8)}
    s["scale"].copy_(scale)
    s["zero"].copy_(zero)
    return s


def _handle(st):
    """The library's cache object over the same tensors."""
    import paged_kv_cache_num_gb300 as pkv
    k, v = st["k"], st["v"]
    return pkv.KVCache("u4", k["data"], v["data"], k_qscale=k["scale"], k_qzero=k["zero"], v_qscale=v["scale"], v_qzero=v["zero"])


def _slots(c, P, g):
    """Slots of tokens that fill blocks drawn from the pool in random order."""
    T, BS = c["tokens"], c["block"]
    blocks = torch.randperm(P, generator=g, device=DEV)[:-(-T // BS)]
    i = torch.arange(T, device=DEV)
    return blocks[i // BS] * BS + i % BS


def _prepare_attention(c, g, st):
    new, ctx = _lengths(c)
    need = [-(-t // c["block"]) for t in ctx]
    P = sum(need) + sum(need) // 10 + 1
    st["k"], st["v"] = _half_cache(c, P, g), _half_cache(c, P, g)
    ids = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    bt = torch.zeros((c["batch"], max(need)), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    st["q"] = _randn((starts[-1], c["heads"], c["dim"]), g, DTYPES[c["dtype"]])
    st["block_tables"] = bt
    st["q_starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    st["context_lens"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    st["most_new"], st["most_ctx"] = max(new), max(ctx)
    st["out"] = torch.empty_like(st["q"])
    if own:
        import paged_kv_cache_num_gb300 as pkv
        st["cache"] = _handle(st)
        size = pkv.decode_workspace_bytes if c["op"] == "decode" else pkv.prefill_workspace_bytes
        st["workspace"] = torch.empty(size(st["q"], st["cache"], bt), dtype=torch.uint8, device=DEV)


def _prepare_tables(c, g, st):
    cached, new, kept = _requests(c)
    BS = c["block"]
    have = [-(-t // BS) for t in cached]
    last = [-(-(a + n) // BS) for a, n in zip(cached, new)]
    P = sum(last) + 7
    ids = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    st["block_tables"] = torch.zeros((c["batch"], max(1, max(last))), dtype=torch.int32, device=DEV)
    rows = torch.repeat_interleave(torch.arange(c["batch"]), torch.tensor(have))
    cols = torch.cat([torch.arange(n) for n in have])
    st["block_tables"][rows.to(DEV), cols.to(DEV)] = ids[:sum(have)]
    free = ids[sum(have):]
    st["free_blocks"] = torch.zeros(P, dtype=torch.int32, device=DEV)
    st["free_blocks"][:free.numel()] = free
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    st["free_count"] = i32([free.numel()])
    st["cached"], st["new"], st["kept"] = i32(cached), i32(new), i32(kept)
    N = max(1, -(-sum(new) // 256) * 256)           # rows of the step, filled up for a captured graph
    st["context_lens"], st["kept_lens"] = torch.empty_like(st["cached"]), torch.empty_like(st["cached"])
    st["q_starts"], st["free_left"], st["free_after"] = i32([0] * (c["batch"] + 1)), i32([0]), i32([0])
    st["req"], st["pos"] = i32([0] * N), i32([0] * N)
    st["slots"] = torch.zeros(N, dtype=torch.int64, device=DEV)


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    if c["op"] in ("decode", "prefill"):
        _prepare_attention(c, g, st)
        return st
    if c["op"] == "tables":
        _prepare_tables(c, g, st)
        return st
    T, H, D, dt = c["tokens"], c["kv_heads"], c["dim"], DTYPES[c["dtype"]]
    P = -(-T // c["block"]) * 11 // 10 + 1
    st["slots"] = _slots(c, P, g)
    if c["op"] == "append":
        st["k_new"], st["v_new"] = _randn((T, H, D), g, dt), _randn((T, H, D), g, dt)
        for n in ("k", "v"):
            st[n] = {"data": torch.zeros((P, c["block"], H, D // 2), dtype=torch.uint8, device=DEV),
                     "scale": _head_major(P, c["block"], H, torch.float16), "zero": _head_major(P, c["block"], H, torch.uint8)}
        st["k_out"], st["v_out"] = torch.empty((T, H, D), dtype=dt, device=DEV), torch.empty((T, H, D), dtype=dt, device=DEV)
        if own:
            st["cache"] = _handle(st)
        return st
    # the fused projection's output, [token][q heads | k heads | v heads]
    qkv = _randn((T, c["heads"] + 2 * H, D), g, dt)
    st["q"], st["k_new"], st["v_new"] = qkv.split([c["heads"], H, H], 1)
    st["q_weight"] = (1 + 0.2 * _randn((D,), g)).to(dt) if c["norm"] else None
    st["k_weight"] = (1 + 0.2 * _randn((D,), g)).to(dt) if c["norm"] else None
    half = c["rot"] // 2
    angle = torch.arange(FAR, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
    st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], -1).float()
    st["pos"] = torch.randint(0, FAR, (T,), generator=g, device=DEV, dtype=torch.int32)
    st["q_out"] = torch.empty((T, c["heads"], D), dtype=dt, device=DEV)
    st["k_cache"] = torch.zeros((P, c["block"], H, D), dtype=dt, device=DEV)
    st["v_cache"] = torch.zeros_like(st["k_cache"])
    if own:
        import paged_kv_cache_num_gb300 as pkv
        st["cache"] = pkv.KVCache(c["dtype"], st["k_cache"], st["v_cache"])
    return st


# ---------------------------------------------------------------- plain forms
def _values(half, ids):
    """Blocks or rows `ids` of one of K and V in 32 bits: (code - zero) * scale."""
    b = half["data"][ids]
    codes = torch.stack([b & 15, b >> 4], -1).flatten(-2).float()
    return (codes - half["zero"][ids].float().unsqueeze(-1)) * half["scale"][ids].float().unsqueeze(-1)


def _plain_attention(st):
    c, q = st["case"], st["q"]
    B, n, t = c["batch"], st["most_new"], st["most_ctx"]
    Hkv, D = c["kv_heads"], c["dim"]
    G = c["heads"] // Hkv
    ids = st["block_tables"].long()
    k = _values(st["k"], ids).flatten(1, 2)[:, :t].transpose(1, 2)              # [B, Hkv, t, D]
    v = _values(st["v"], ids).flatten(1, 2)[:, :t].transpose(1, 2)
    start, ctx = st["q_starts"][:-1].long(), st["context_lens"].long()
    new = st["q_starts"][1:].long() - start
    i = torch.arange(n, device=q.device)
    rows = (start[:, None] + i).clamp(max=q.shape[0] - 1)                       # [B, n]
    x = q.float()[rows].view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    s = torch.matmul(x, k.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, G, n, t)
    last = (ctx - new)[:, None] + i                                             # last key that a row sees
    hidden = torch.arange(t, device=q.device) > last[:, :, None]                # [B, n, t]
    s.masked_fill_(hidden[:, None, None], float("-inf"))
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(s.view(B, Hkv, G * n, t), v).view(B, Hkv, G, n, D) / s.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hkv * G, D)
    tok = torch.arange(q.shape[0], device=q.device)
    seq = torch.searchsorted(st["q_starts"][1:].long(), tok, right=True)
    return o[seq, tok - start[seq]].to(q.dtype)


def _plain_append(st):
    BS, dt = st["case"]["block"], DTYPES[st["case"]["dtype"]]
    at = (st["slots"] // BS, st["slots"] % BS)
    out = {}
    for n in ("k", "v"):
        half = st[n]
        codes, half["scale"][at], half["zero"][at] = _row_codes(st[n + "_new"].float())
        half["data"][at] = _pack4(codes)
        out[n] = _values(half, at).to(dt)
    return out


def _plain_norm_rope(x, weight, cos, sin, pairs):
    """Rows [T, H, D] in 32 bits, normed and rotated."""
    x = x.float()
    if weight is not None:
        x = x / ((x * x).mean(-1, keepdim=True) + EPS).sqrt() * weight.float()
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if pairs else (x[..., :half], x[..., half:2 * half])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_rope(st):
    c = st["case"]
    dt, at = DTYPES[c["dtype"]], (st["slots"] // c["block"], st["slots"] % c["block"])
    cos, sin = st["cos_sin"][st["pos"].long()].unsqueeze(1).chunk(2, -1)
    q = _plain_norm_rope(st["q"], st["q_weight"], cos, sin, c["pairs"]).to(dt)
    st["k_cache"][at] = _plain_norm_rope(st["k_new"], st["k_weight"], cos, sin, c["pairs"]).to(dt)
    st["v_cache"][at] = st["v_new"]
    return {"q": q, "k": st["k_cache"], "v": st["v_cache"]}


def _plain_tables(st):
    BS, bt, N = st["case"]["block"], st["block_tables"], st["slots"].shape[0]
    cached, new = st["cached"].long(), st["new"].long()
    ctx = cached + new
    have = (cached + BS - 1) // BS
    need = (ctx + BS - 1) // BS - have
    ends = need.cumsum(0)
    first = ends - need                                                         # blocks handed out to those before
    count = st["free_count"].long()
    col = torch.arange(bt.shape[1], device=DEV)
    i = col - have[:, None]
    fresh = (i >= 0) & (i < need[:, None])
    at = (count - 1 - (first[:, None] + i)).clamp(min=0, max=st["free_blocks"].shape[0] - 1)
    bt.copy_(torch.where(fresh, st["free_blocks"][at], bt))
    rows = new.cumsum(0)
    starts = torch.cat([rows.new_zeros(1), rows])
    r = torch.arange(N, device=DEV)
    b = torch.searchsorted(rows, r, right=True)
    live = b < new.shape[0]
    b = b.clamp(max=new.shape[0] - 1)
    pos = cached[b] + r - starts[b]
    slots = bt[b, (pos // BS).clamp(max=bt.shape[1] - 1)].long() * BS + pos % BS
    left = count - ends[-1:]
    out = {"block_tables": bt, "context_lens": ctx.int(), "q_starts": starts.int(), "req": torch.where(live, b, -1).int(),
           "pos": torch.where(live, pos, -1).int(), "slots": torch.where(live, slots, -1), "free_left": left.int()}
    if st["case"]["trim"]:
        keep = torch.minimum(st["kept"].long(), ctx)
        have, stay = (ctx + BS - 1) // BS, (keep + BS - 1) // BS
        drop = have - stay
        ends = drop.cumsum(0)
        i = col - stay[:, None]
        gone = (i >= 0) & (i < drop[:, None])
        free = st["free_blocks"].clone()
        room = torch.cat([free, free.new_zeros(1)])                             # the last entry takes what is kept
        at = torch.where(gone, left + (ends - drop)[:, None] + i, free.shape[0])
        room[at] = bt
        out |= {"kept_lens": keep.int(), "free_blocks": room[:-1], "free_after": (left + ends[-1:]).int()}
    return out


def run(state):
    st, c = state, state["case"]
    op = c["op"]
    if not own:
        return (_plain_append if op == "append" else _plain_rope if op == "rope" else _plain_tables if op == "tables" else _plain_attention)(st)
    import paged_kv_cache_num_gb300 as pkv
    if op == "decode":
        return pkv.paged_decode(st["q"], st["cache"], st["block_tables"], st["context_lens"], out=st["out"], workspace=st["workspace"])
    if op == "prefill":
        return pkv.paged_prefill(st["q"], st["cache"], st["block_tables"], st["q_starts"], st["context_lens"], out=st["out"], workspace=st["workspace"])
    if op == "append":
        pkv.kv_append(st["k_new"], st["v_new"], st["slots"], st["cache"])
        k, v = pkv.kv_gather(st["cache"], st["slots"], k_out=st["k_out"], v_out=st["v_out"])
        return {"k": k, "v": v}
    if op == "rope":
        q = pkv.norm_rope_append(st["q"], st["k_new"], st["v_new"], st["cos_sin"], st["pos"], st["slots"], st["cache"], q_weight=st["q_weight"],
                                 k_weight=st["k_weight"], eps=EPS, interleaved=c["pairs"], q_out=st["q_out"])
        return {"q": q, "k": st["k_cache"], "v": st["v_cache"]}
    ctx, starts, req, pos, slots, left = pkv.extend_tables(
        st["block_tables"], st["cached"], st["new"], st["free_blocks"], st["free_count"], c["block"], context_lens=st["context_lens"],
        q_starts=st["q_starts"], req=st["req"], pos=st["pos"], slot_mapping=st["slots"], free_left=st["free_left"])
    out = {"block_tables": st["block_tables"], "context_lens": ctx, "q_starts": starts, "req": req, "pos": pos, "slots": slots, "free_left": left}
    if c["trim"]:
        free = st["free_blocks"].clone()                # what comes back is pushed on it; this case starts from the same blocks each time
        kept, after = pkv.trim_tables(st["block_tables"], ctx, st["kept"], free, left, c["block"], kept_lens=st["kept_lens"], free_left=st["free_after"])
        out |= {"kept_lens": kept, "free_blocks": free, "free_after": after}
    return out


# ---------------------------------------------------------------- work and the 64-bit result
def work(case):
    c = case
    if c["op"] == "tables":
        cached, new, _ = _requests(c)
        BS = c["block"]
        fresh = sum(-(-(a + n) // BS) - -(-a // BS) for a, n in zip(cached, new))
        N = max(1, -(-sum(new) // 256) * 256)
        return {"bytes": c["batch"] * (16 if c["trim"] else 12) + fresh * (16 if c["trim"] else 8) + N * 16, "flops": 0}
    D, H = c["dim"], c["kv_heads"]
    row = D // 2 + 3                                # a cached row with its scale and zero
    if c["op"] == "append":
        return {"bytes": c["tokens"] * (2 * H * (2 * D + row + 2 * D) + 8), "flops": c["tokens"] * 2 * H * D * 6}
    if c["op"] == "rope":
        heads = c["heads"] + 2 * H
        return {"bytes": c["tokens"] * (heads * 4 * D + 4 * c["rot"] + 12), "flops": c["tokens"] * (c["heads"] + H) * D * 7}
    new, ctx = _lengths(c)
    pairs = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(new, ctx))
    blocks = sum(-(-t // c["block"]) for t in ctx)
    return {"bytes": sum(new) * c["heads"] * D * 4 + sum(ctx) * 2 * H * row + blocks * 4 + c["batch"] * 8, "flops": 4 * D * c["heads"] * pairs}


def _exact_rows(half, blk, off):
    """Rows at (blk, off) [...] as float64, from the format's definition: element d is bits 4d .. 4d + 3."""
    raw = half["data"][blk, off]
    bits = torch.stack([(raw >> i) & 1 for i in range(8)], -1).flatten(-2)
    x = sum(bits[..., i::4].double() * 2 ** i for i in range(4))
    return (x - half["zero"][blk, off].double()[..., None]) * half["scale"][blk, off].double()[..., None]


def _exact_attention(case, st):
    c, BS = case, case["block"]
    new, ctx = _lengths(c)
    q, G, D = st["q"].double(), c["heads"] // c["kv_heads"], c["dim"]
    if 4 * D * c["heads"] * sum(n * t for n, t in zip(new, ctx)) > 6e12:
        return None
    out = torch.empty_like(q)
    at = 0
    for b, (n, t) in enumerate(zip(new, ctx)):
        pos = torch.arange(t, device=q.device)
        blk, off = st["block_tables"][b].long()[pos // BS], pos % BS
        k, v = _exact_rows(st["k"], blk, off), _exact_rows(st["v"], blk, off)           # [t, H, D]
        seen = pos[None] <= (t - n + torch.arange(n, device=q.device))[:, None]         # [n, t]
        for h in range(c["kv_heads"]):
            s = torch.einsum("ngd,td->gnt", q[at:at + n, h * G:(h + 1) * G], k[:, h]) / math.sqrt(D)
            p = torch.softmax(torch.where(seen, s, -math.inf), -1)
            out[at:at + n, h * G:(h + 1) * G] = torch.einsum("gnt,td->ngd", p, v[:, h])
        at += n
    return out


def _exact_turn(x, weight, angle, pairs):
    x = x.double()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.double()
    half = angle.shape[-1] // 2
    turn = torch.complex(*angle.double()[:, None].split(half, -1))                      # e^(i angle) as the table has it
    y = x.clone()
    i = torch.arange(half, device=x.device)
    re, im = (2 * i, 2 * i + 1) if pairs else (i, i + half)
    z = torch.complex(x[..., re], x[..., im]) * turn
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_tables(case, st):
    """Block by block and token by token, as a host would."""
    BS = case["block"]
    cached, new, kept = _requests(case)
    bt = st["block_tables"].cpu().clone()
    stack = st["free_blocks"][:int(st["free_count"])].tolist()
    starts, req, pos, ctx = [0], [], [], []
    for b, (a, n) in enumerate(zip(cached, new)):
        for j in range(-(-a // BS), -(-(a + n) // BS)):
            bt[b, j] = stack.pop()
        starts.append(starts[-1] + n)
        req += [b] * n
        pos += range(a, a + n)
        ctx.append(a + n)
    N = st["slots"].shape[0]
    r, p = torch.tensor(req, dtype=torch.long), torch.tensor(pos, dtype=torch.long)
    slots = torch.full((N,), -1)
    slots[:len(req)] = bt[r, p // BS].long() * BS + p % BS
    fill = lambda x: torch.tensor(x + [-1] * (N - len(x)), dtype=torch.int32)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    out = {"block_tables": bt, "context_lens": i32(ctx), "q_starts": i32(starts), "req": fill(req), "pos": fill(pos), "slots": slots,
           "free_left": i32([len(stack)])}
    if case["trim"]:
        free = st["free_blocks"].cpu().clone()
        keep = [min(k, t) for k, t in zip(kept, ctx)]
        at = len(stack)
        for b, (k, t) in enumerate(zip(keep, ctx)):
            for j in range(-(-k // BS), -(-t // BS)):
                free[at] = bt[b, j]
                at += 1
        out |= {"kept_lens": i32(keep), "free_blocks": free, "free_after": i32([at])}
    return {n: t.to(DEV) for n, t in out.items()}


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] in ("decode", "prefill"):
        return _exact_attention(c, st)
    if c["op"] == "tables":
        return _exact_tables(c, st)
    if c["op"] == "append":
        out = {}
        for n in ("k", "v"):
            x = st[n + "_new"].double()
            zero = torch.zeros_like(x[..., :1])
            span = torch.cat([x, zero], -1)
            lo = span.min(-1, keepdim=True).values
            # a stored scale has 16 bits, and the quotients that are rounded have 32
            s = ((span.max(-1, keepdim=True).values - lo) / 15).float().half().double()
            steps = lambda y: torch.where(s > 0, (y / s).float().double().round(), zero)  # noqa: E731
            z = steps(-lo).clamp(0, 15)
            out[n] = ((steps(x) + z).clamp(0, 15) - z) * s
        return out
    blk, off = st["slots"] // c["block"], st["slots"] % c["block"]
    angle = st["cos_sin"][st["pos"].long()]
    k, v = st["k_cache"].double(), st["v_cache"].double()
    k[blk, off] = _exact_turn(st["k_new"], st["k_weight"], angle, c["pairs"])
    v[blk, off] = st["v_new"].double()
    return {"q": _exact_turn(st["q"], st["q_weight"], angle, c["pairs"]), "k": k, "v": v}
