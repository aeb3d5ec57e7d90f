"""Cases of the cache's prompt-side operators: attention of packed new tokens
over the paged cache (paged_prefill), the append that computes its own
per-token scales (kv_append_dynamic) and the read back of cached rows
(kv_gather).

A case is a dict of plain values; prepare() makes the inputs on the GPU from
a seed, run() makes one pass (the plain form in elementary torch operations,
or the library's call where `own` is set), exact() gives the result in 64
bits, work() what a pass has to move and compute.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
QMAX = {"e4m3": 448.0, "e5m2": 57344.0, "i8": 127.0}
CODE_DTYPES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "i8": torch.int8}
TINY = 2.0 ** -126                   # least scale of a row


# ---------------------------------------------------------------- cases
def listed():
    pre = {"op": "prefill", "layout": "flash", "scales": "head", "dtype": "bf16", "dim": 128, "block": 16}
    app = {"op": "append", "layout": "flash", "dim": 128, "block": 16, "dtype": "bf16", "kv_heads": 8}
    gat = {"op": "gather", "layout": "flash", "scales": "token", "dim": 128, "block": 16, "dtype": "bf16", "kv_heads": 8}
    return [
        # one short chat turn: a single prompt of a few dozen tokens, where latency counts
        dict(pre, name="prefill_short", kind="bf16", heads=32, kv_heads=8, batch=1, new_lo=37, new_hi=37, ctx_lo=0, ctx_hi=0, mix=1),
        # a serving batch of whole prompts of very different lengths, packed
        dict(pre, name="prefill_packed", kind="bf16", heads=32, kv_heads=8, batch=16, new_lo=60, new_hi=1500, ctx_lo=0, ctx_hi=0, mix=2),
        # one long document in a single pass
        dict(pre, name="prefill_long", kind="bf16", heads=32, kv_heads=8, batch=1, new_lo=12001, new_hi=12001, ctx_lo=0, ctx_hi=0, mix=3),
        # chunked prefill over long fp8 contexts with the headline decode's head layout
        dict(pre, name="prefill_chunks_e4m3", kind="e4m3", heads=64, kv_heads=8, block=32, batch=4, new_lo=400, new_hi=512, ctx_lo=8192, ctx_hi=16384, mix=4),
        # a few drafted tokens per sequence checked over paged contexts
        dict(pre, name="prefill_draft_few", kind="bf16", heads=32, kv_heads=8, batch=32, new_lo=1, new_hi=8, ctx_lo=512, ctx_hi=4096, mix=5),
        # multi-head model with the 3-bit cache, chunks of prompts
        dict(pre, name="prefill_chunks_u3", kind="u3", dtype="f16", heads=32, kv_heads=32, batch=8, new_lo=100, new_hi=300, ctx_lo=1024, ctx_hi=4096, mix=6),
        # one decode step's tokens, quantised as they are written
        dict(app, name="append_step_e4m3", kind="e4m3", tokens=64),
        # a prefill's worth of tokens into an int8 cache
        dict(app, name="append_prompt_i8", kind="i8", dtype="f16", tokens=60001),
        # odd head count and length, x-vectorised storage
        dict(app, name="append_odd_e5m2", kind="e5m2", layout="xvec", dim=64, kv_heads=5, tokens=1777),
        # a few blocks of one sequence read back
        dict(gat, name="gather_few_e4m3", kind="e4m3", tokens=200),
        # a long context moved out of a per-token-scale fp8 cache
        dict(gat, name="gather_long_e4m3", kind="e4m3", tokens=100003),
        # 3-bit multi-head context read back
        dict(gat, name="gather_u3", kind="u3", scales="head", dtype="f16", kv_heads=32, tokens=20001),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "append", "gather"])
    dtype, dim = rng.choice(["bf16", "f16"]), rng.choice([64, 128, 128])
    case = {"op": op, "dtype": dtype, "dim": dim, "block": rng.choice([8, 16, 16, 32, 64]), "layout": rng.choice(["flash", "flash", "xvec"])}
    if op == "append":
        kind, heads = rng.choice(["e4m3", "e5m2", "i8"]), rng.randint(1, 16)
        case |= {"kind": kind, "kv_heads": heads, "tokens": _log_int(rng, 1, 480000 // heads)}
        return case
    kind = rng.choice([dtype, dtype, "e4m3", "e5m2", "i8", "u3"])
    case["kind"] = kind
    case["scales"] = rng.choice(["head", "block", "token"]) if kind in QMAX else "head"
    if kind == "u3":
        case["layout"] = "flash"
    if op == "gather":
        heads = rng.randint(1, 32)
        case |= {"kv_heads": heads, "tokens": _log_int(rng, 1, 400000 // heads)}
        return case
    kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    batch = _log_int(rng, 1, 48)
    new_hi = _log_int(rng, 1, max(2, 6000 // batch))
    new_lo = rng.randint(1, new_hi)
    ctx_hi = rng.choice([0, _log_int(rng, new_hi, 8192)])
    # no more query-key pairs than the long document's
    while batch * kv * group * new_hi * max(new_hi, ctx_hi) > 1.2e9:
        batch, new_hi = max(1, batch // 2), max(1, new_hi * 3 // 4)
        new_lo = min(new_lo, new_hi)
    case |= {"heads": kv * group, "kv_heads": kv, "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "ctx_lo": ctx_hi // 4, "ctx_hi": ctx_hi,
             "mix": rng.randint(1, 10 ** 6)}
    return case


def _lengths(c):
    """(new tokens, context length) of each sequence of a prefill case."""
    r = random.Random(c["mix"])
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["batch"])]
    return new, [max(n, r.randint(c["ctx_lo"], c["ctx_hi"])) for n in new]


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _to_codes(x, scale, kind):
    y = x / scale
    if kind == "i8":
        return y.round().clamp(-127, 127).to(torch.int8)
    return y.clamp(-QMAX[kind], QMAX[kind]).to(CODE_DTYPES[kind])


def _xvec(t, x):
    """[P, BS, H, D] -> the x-vectorised storage [P, H, D / x, BS, x]."""
    P, BS, H, D = t.shape
    return t.view(P, BS, H, D // x, x).permute(0, 2, 3, 1, 4).contiguous()


def _pack3(codes):
    """[..., D] codes of 3 bits -> [..., 3 D / 8] bytes, little-endian bit string."""
    o = codes.view(*codes.shape[:-1], -1, 8).to(torch.int32)
    w = (o << (3 * torch.arange(8, device=o.device, dtype=torch.int32))).sum(-1, dtype=torch.int32)
    b = torch.stack([w & 255, (w >> 8) & 255, (w >> 16) & 255], -1)
    return b.to(torch.uint8).flatten(-2)


def _half_cache(c, P, g):
    """One of K and V: {"data", and what its kind needs}."""
    BS, H, D, kind = c["block"], c["kv_heads"], c["dim"], c["kind"]
    x = _randn((P, BS, H, D), g)
    s = {}
    if kind == "u3":
        lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
        qs = ((hi - lo) / 7).to(torch.float16)
        z = (-lo / qs.float()).round().clamp(0, 7)
        data = _pack3(((x / qs.float()).round() + z).clamp(0, 7).to(torch.uint8))
        # scale and zero kept head by head behind a [P, BS, H] view, as the library allocates them
        s["qscale"] = qs[..., 0].transpose(1, 2).contiguous().transpose(1, 2)
        s["qzero"] = z[..., 0].to(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2)
    elif kind in QMAX:
        if c["scales"] == "head":
            s["scale"] = x.abs().amax((0, 1, 3)) / QMAX[kind]
            sc = s["scale"].view(1, 1, H, 1)
        elif c["scales"] == "block":
            s["scales"] = x.abs().amax((1, 3)) / QMAX[kind]
            sc = s["scales"].view(P, 1, H, 1)
        else:
            s["scales"] = (x.abs().amax(3) / QMAX[kind]).transpose(1, 2).contiguous().transpose(1, 2)
            sc = s["scales"].unsqueeze(-1)
        data = _to_codes(x, sc, kind)
        data = data if kind == "i8" else data.view(torch.uint8)
    else:
        data = x.to(DTYPES[kind])
    s["data"] = _xvec(data, 16 // data.element_size()) if c["layout"] == "xvec" else data
    return s


def _handle(st, c):
    """The library's cache object over the same tensors."""
    import paged_kv_cache_num_gb300 as pkv
    k, v = st["k"], st["v"]
    return pkv.KVCache(c["kind"], k["data"], v["data"], k_scale=k.get("scale"), v_scale=v.get("scale"), k_qscale=k.get("qscale"), k_qzero=k.get("qzero"),
                       v_qscale=v.get("qscale"), v_qzero=v.get("qzero"), scale_mode=c.get("scales", "head"), k_scales=k.get("scales"), v_scales=v.get("scales"),
                       layout=c["layout"])


def _slots(c, P, g):
    """Slots of tokens that fill blocks drawn from the pool in random order."""
    T, BS = c["tokens"], c["block"]
    blocks = torch.randperm(P, generator=g, device=DEV)[:-(-T // BS)]
    i = torch.arange(T, device=DEV)
    return blocks[i // BS] * BS + i % BS


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    dt = DTYPES[c["dtype"]]
    if c["op"] == "prefill":
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
        st["q"] = _randn((starts[-1], c["heads"], c["dim"]), g, dt)
        st["block_tables"] = bt
        st["q_starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        st["context_lens"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        st["most_new"], st["most_ctx"] = max(new), max(ctx)
        st["out"] = torch.empty_like(st["q"])
        if own:
            import paged_kv_cache_num_gb300 as pkv
            st["cache"] = _handle(st, c)
            st["workspace"] = torch.empty(pkv.prefill_workspace_bytes(st["q"], st["cache"], bt), dtype=torch.uint8, device=DEV)
        return st
    P = -(-c["tokens"] // c["block"]) * 11 // 10 + 1
    if c["op"] == "append":
        H, D = c["kv_heads"], c["dim"]
        c = dict(c, scales="token")
        st["k_new"] = _randn((c["tokens"], H, D), g, dt)
        st["v_new"] = _randn((c["tokens"], H, D), g, dt)
        shape = (P, H, D // 16, c["block"], 16) if c["layout"] == "xvec" else (P, c["block"], H, D)
        for n in ("k", "v"):
            st[n] = {"data": torch.zeros(shape, dtype=torch.int8 if c["kind"] == "i8" else torch.uint8, device=DEV),
                     "scales": torch.ones((P, H, c["block"]), device=DEV).transpose(1, 2)}
    else:
        st["k"], st["v"] = _half_cache(c, P, g), _half_cache(c, P, g)
        st["k_out"] = torch.empty((c["tokens"], c["kv_heads"], c["dim"]), dtype=dt, device=DEV)
        st["v_out"] = torch.empty_like(st["k_out"])
    st["slots"] = _slots(c, P, g)
    if own:
        st["cache"] = _handle(st, c)
    return st


# ---------------------------------------------------------------- plain forms
def _unpack3(packed):
    """[..., 3 D / 8] bytes -> [..., D] codes."""
    b = packed.view(*packed.shape[:-1], -1, 3).to(torch.int32)
    w = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
    return ((w.unsqueeze(-1) >> (3 * torch.arange(8, device=b.device, dtype=torch.int32))) & 7).flatten(-2)


def _values(rows, kind):
    """Stored rows [..., row] -> their codes or elements in 32 bits."""
    if kind == "u3":
        return _unpack3(rows).float()
    if kind in ("e4m3", "e5m2"):
        return rows.view(CODE_DTYPES[kind]).float()
    return rows.float()


def _blocks(half, ids, c):
    """Whole blocks `ids` [...] in 32 bits, dequantised: [..., BS, H, D]."""
    data = half["data"][ids]
    if c["layout"] == "xvec":                       # [..., H, C, BS, x] -> [..., BS, H, C, x]
        n = data.dim()
        data = data.permute(*range(n - 4), n - 2, n - 4, n - 3, n - 1).flatten(-2)
    x = _values(data, c["kind"])
    if c["kind"] == "u3":
        return (x - half["qzero"][ids].float().unsqueeze(-1)) * half["qscale"][ids].float().unsqueeze(-1)
    if c["kind"] in QMAX:
        if c["scales"] == "head":
            return x * half["scale"].view(-1, 1)
        s = half["scales"][ids]
        return x * (s.unsqueeze(-2) if c["scales"] == "block" else s).unsqueeze(-1)
    return x


def _plain_prefill(st):
    c, q = st["case"], st["q"]
    B, n, t = c["batch"], st["most_new"], st["most_ctx"]
    Hkv, D = c["kv_heads"], c["dim"]
    G = c["heads"] // Hkv
    ids = st["block_tables"].long()
    k = _blocks(st["k"], ids, c).flatten(1, 2)[:, :t].transpose(1, 2)           # [B, Hkv, t, D]
    v = _blocks(st["v"], ids, c).flatten(1, 2)[:, :t].transpose(1, 2)
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
    c = st["case"]
    BS = c["block"]
    blk, off = st["slots"] // BS, st["slots"] % BS
    out = {}
    for n in ("k", "v"):
        x, half = st[n + "_new"].float(), st[n]
        top = x.abs().amax(-1)
        # divided by a tensor: by a Python number it would be a product with the reciprocal
        scale = (top / torch.full((), QMAX[c["kind"]], device=top.device)).clamp(min=TINY)
        codes = _to_codes(x, scale.unsqueeze(-1), c["kind"])
        codes = codes if c["kind"] == "i8" else codes.view(torch.uint8)
        if c["layout"] == "xvec":                                               # storage [P, H, C, BS, x]
            half["data"].permute(0, 3, 1, 2, 4)[blk, off] = codes.view(*codes.shape[:-1], -1, 16)
        else:
            half["data"][blk, off] = codes
        half["scales"][blk, off] = scale
        out[n], out[n + "_scales"] = half["data"].view(CODE_DTYPES[c["kind"]]), half["scales"]
    return out


def _plain_gather(st):
    c = st["case"]
    BS = c["block"]
    blk, off = st["slots"] // BS, st["slots"] % BS
    out = {}
    for n in ("k", "v"):
        half = st[n]
        data = half["data"].permute(0, 3, 1, 2, 4)[blk, off].flatten(-2) if c["layout"] == "xvec" else half["data"][blk, off]
        x = _values(data, c["kind"])
        if c["kind"] == "u3":
            x = (x - half["qzero"][blk, off].float().unsqueeze(-1)) * half["qscale"][blk, off].float().unsqueeze(-1)
        elif c["kind"] in QMAX:
            s = half["scale"] if c["scales"] == "head" else half["scales"][blk] if c["scales"] == "block" else half["scales"][blk, off]
            x = x * s.unsqueeze(-1)
        out[n] = x.to(DTYPES[c["dtype"]])
    return out


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        import paged_kv_cache_num_gb300 as pkv
        if op == "prefill":
            return pkv.paged_prefill(st["q"], st["cache"], st["block_tables"], st["q_starts"], st["context_lens"], out=st["out"], workspace=st["workspace"])
        if op == "append":
            pkv.kv_append_dynamic(st["k_new"], st["v_new"], st["slots"], st["cache"])
            code = CODE_DTYPES[st["case"]["kind"]]
            return {"k": st["k"]["data"].view(code), "k_scales": st["k"]["scales"], "v": st["v"]["data"].view(code), "v_scales": st["v"]["scales"]}
        k, v = pkv.kv_gather(st["cache"], st["slots"], k_out=st["k_out"], v_out=st["v_out"])
        return {"k": k, "v": v}
    return _plain_prefill(st) if op == "prefill" else _plain_append(st) if op == "append" else _plain_gather(st)


# ---------------------------------------------------------------- work and the 64-bit result
def _row_bytes(kind, dim):
    """Bytes of one cached row of one of K and V, with its own scale and zero (3-bit)."""
    return 3 * dim // 8 + 3 if kind == "u3" else dim if kind in QMAX else 2 * dim


def work(case):
    c = case
    D, H = c["dim"], c["kv_heads"]
    if c["op"] == "append":
        return {"bytes": c["tokens"] * (2 * H * (2 * D + D + 4) + 8), "flops": c["tokens"] * 2 * H * D * 3}
    row = _row_bytes(c["kind"], D) + (4 if c["scales"] == "token" else 0)
    if c["op"] == "gather":
        return {"bytes": c["tokens"] * (2 * H * (row + 2 * D) + 8), "flops": 0 if c["kind"] in DTYPES else c["tokens"] * 2 * H * D}
    new, ctx = _lengths(c)
    pairs = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(new, ctx))
    blocks = sum(-(-t // c["block"]) for t in ctx)
    return {"bytes": sum(new) * c["heads"] * D * 4 + sum(ctx) * 2 * H * row + blocks * 4 + c["batch"] * 12, "flops": 4 * D * c["heads"] * pairs}


def _exact_rows(half, blk, off, c):
    """Rows at (blk, off) [...] as float64, from the formats' definitions."""
    raw = half["data"]
    raw = torch.stack([raw[blk, :, j, off] for j in range(raw.shape[2])], -2).flatten(-2) if c["layout"] == "xvec" else raw[blk, off]
    if c["kind"] == "u3":
        bits = torch.stack([(raw >> i) & 1 for i in range(8)], -1).flatten(-2)      # element d: bits 3d .. 3d+2
        x = (bits[..., 0::3] + 2 * bits[..., 1::3] + 4 * bits[..., 2::3]).double()
        return (x - half["qzero"][blk, off].double()[..., None]) * half["qscale"][blk, off].double()[..., None]
    if c["kind"] not in QMAX:
        return raw.double()
    x = raw.double() if c["kind"] == "i8" else raw.view(CODE_DTYPES[c["kind"]]).double()
    if c["scales"] == "head":
        s = half["scale"].double().expand(x.shape[:-1])
    elif c["scales"] == "block":
        s = half["scales"].double()[blk]
    else:
        s = half["scales"].double()[blk, off]
    return x * s[..., None]


def exact(case, seed):
    st, c = prepare(case, seed), case
    BS = c["block"]
    if c["op"] == "gather":
        blk, off = st["slots"] // BS, st["slots"] % BS
        return {n: _exact_rows(st[n], blk, off, c) for n in ("k", "v")}
    if c["op"] == "append":
        out = {}
        for n in ("k", "v"):
            x = st[n + "_new"].double()
            top = x.abs().max(-1).values
            scale = (top / QMAX[c["kind"]]).float().clamp(min=TINY)                 # a stored scale has 32 bits, and
            y = (x / scale.double()[..., None]).float()                             # so has the quotient that is cast
            if c["kind"] == "i8":
                codes = torch.round(y.double()).clamp(-127, 127).to(torch.int8)
            else:
                codes = y.clamp(-QMAX[c["kind"]], QMAX[c["kind"]]).to(CODE_DTYPES[c["kind"]]).double()
            pool = torch.zeros(st[n]["data"].shape, dtype=codes.dtype, device=codes.device)
            for j in range(pool.shape[2] if c["layout"] == "xvec" else 0):
                pool[st["slots"] // BS, :, j, st["slots"] % BS] = codes[..., 16 * j:16 * j + 16]
            if c["layout"] != "xvec":
                pool.view(-1, *pool.shape[2:])[st["slots"]] = codes
            sc = torch.ones(st[n]["scales"].shape, dtype=torch.float64, device=codes.device)
            sc.view(-1, sc.shape[-1])[st["slots"]] = (top / QMAX[c["kind"]]).clamp(min=TINY)
            out[n], out[n + "_scales"] = pool, sc
        return out
    new, ctx = _lengths(c)
    q, H, D = st["q"].double(), c["kv_heads"], c["dim"]
    G = c["heads"] // H
    if 4 * D * c["heads"] * sum(n * t for n, t in zip(new, ctx)) > 6e12:
        return None
    out = torch.empty_like(q)
    at = 0
    for b, (n, t) in enumerate(zip(new, ctx)):
        pos = torch.arange(t, device=q.device)
        blk, off = st["block_tables"][b].long()[pos // BS], pos % BS
        k, v = _exact_rows(st["k"], blk, off, c), _exact_rows(st["v"], blk, off, c)     # [t, H, D]
        step = max(1, int(2e8 // t))
        for h in range(c["heads"]):
            for i in range(0, n, step):
                j = min(n, i + step)
                s = q[at + i:at + j, h] @ k[:, h // G].T / math.sqrt(D)
                seen = pos[None] <= (t - n + torch.arange(i, j, device=q.device))[:, None]
                p = torch.softmax(torch.where(seen, s, -math.inf), -1)
                out[at + i:at + j, h] = p @ v[:, h // G]
        at += n
    return out
