"""The 8-bit paged KV cache: what is measured of awq_rope_table, awq_kv8_append and
awq_attn_kv8, with their plain forms in elementary torch operations.

A decode or prefill step of a decoder layer runs its q, k and v projections, then
rotates q and k by position, appends k and v to the cache, attends over the cache and
goes on with the o projection.  The cache is paged: page `j` of sequence `b` is
block_table[b][j], holding `page` tokens of every key/value head in e4m3 codes with one
float32 scale per page and head (keys and values apart):

  k_cache [pages][hkv][page][d], v_cache [pages][hkv][d][page], k_scale, v_scale [pages][hkv]

New tokens are the rows cu_q[b] .. cu_q[b+1]-1 of q, k and v (cu_q None: one per
sequence); ctx[b] counts the sequence's tokens with the new ones, so new token i of n
stands at position ctx[b] - n + i and sees positions 0 .. ctx[b] - n + i.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
FP8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the table of a short context, and of a 128 K context with frequencies scaled by bands
        {"name": "table_8k", "op": "table", "positions": 8192, "rot": 128, "base": 500000.0, "scaling": "none"},
        {"name": "table_128k_bands", "op": "table", "positions": 131072, "rot": 128, "base": 500000.0,
         "scaling": "bands"},
        # one sequence's decode step; a batch of 64 ragged ones (70B-shaped heads); packed prompts;
        # rotation of a quarter of a 64-wide head in the interleaved layout, with idle sequences
        {"name": "append_decode_1", "op": "append", "dtype": "fp16", "b": 1, "new": 1, "past": 700, "hq": 32,
         "hkv": 8, "d": 128, "page": 64, "rot": 128, "inter": False, "pad": 0, "mix": 1},
        {"name": "append_decode_64", "op": "append", "dtype": "bf16", "b": 64, "new": 1, "past": 4096, "hq": 64,
         "hkv": 8, "d": 128, "page": 64, "rot": 128, "inter": False, "pad": 0, "mix": 2},
        {"name": "append_prompts", "op": "append", "dtype": "fp16", "b": 7, "new": 2048, "past": 0, "hq": 32,
         "hkv": 8, "d": 128, "page": 64, "rot": 128, "inter": False, "pad": 37, "mix": 3},
        {"name": "append_part_d64", "op": "append", "dtype": "bf16", "b": 33, "new": 9, "past": 1500, "hq": 24,
         "hkv": 6, "d": 64, "page": 128, "rot": 16, "inter": True, "pad": 5, "mix": 4},
        # decode attention: one short sequence (latency), a ragged batch, 64 long ones with
        # 70B-shaped heads, one sequence of 128 K tokens
        {"name": "attn_decode_1", "op": "attn", "dtype": "fp16", "b": 1, "new": 1, "past": 700, "hq": 32, "hkv": 8,
         "d": 128, "page": 64, "pad": 0, "mix": 5},
        {"name": "attn_decode_64", "op": "attn", "dtype": "bf16", "b": 64, "new": 1, "past": 8191, "hq": 64,
         "hkv": 8, "d": 128, "page": 64, "pad": 0, "mix": 6},
        {"name": "attn_decode_128k", "op": "attn", "dtype": "fp16", "b": 1, "new": 1, "past": 131071, "hq": 32,
         "hkv": 8, "d": 128, "page": 64, "pad": 0, "mix": 7},
        # a few tokens per sequence (a draft being verified), odd counts, 64-wide heads
        {"name": "attn_verify_d64", "op": "attn", "dtype": "bf16", "b": 19, "new": 5, "past": 3001, "hq": 24, "hkv": 6,
         "d": 64, "page": 128, "pad": 3, "mix": 8},
        # a whole prompt, and chunks of different prompts behind earlier context
        {"name": "attn_prompt_8k", "op": "attn", "dtype": "bf16", "b": 1, "new": 8192, "past": 0, "hq": 32, "hkv": 8,
         "d": 128, "page": 64, "pad": 0, "mix": 9},
        {"name": "attn_chunks", "op": "attn", "dtype": "fp16", "b": 5, "new": 777, "past": 6000, "hq": 32, "hkv": 8,
         "d": 128, "page": 64, "pad": 11, "mix": 10},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("table", "append", "append", "attn", "attn", "attn"))
    if op == "table":
        return {"op": "table", "positions": _log(rng, 500, 131072), "rot": rng.choice((16, 32, 64, 96, 128)),
                "base": rng.choice((10000.0, 500000.0)), "scaling": rng.choice(("none", "linear", "bands", "yarn"))}
    hkv = rng.choice((1, 2, 4, 6, 8, 8, 32))
    hq = hkv * (1 if hkv == 32 else rng.choice((1, 2, 3, 4, 4, 7, 8)))
    d = rng.choice((64, 128, 128))
    c = {"op": op, "dtype": rng.choice(("fp16", "bf16")), "hq": hq, "hkv": hkv, "d": d,
         "page": rng.choice((64, 64, 128, 256)), "pad": rng.choice((0, 0, 0, 9)), "mix": rng.randrange(1 << 20)}
    kind = rng.choice(("decode", "decode", "verify", "prompt"))
    if kind == "decode":
        c.update(b=_log(rng, 1, 64), new=1, past=_log(rng, 1, 16384))
    elif kind == "verify":
        c.update(b=_log(rng, 1, 32), new=rng.randrange(2, 10), past=_log(rng, 1, 8192))
    else:
        c.update(b=rng.randrange(1, 6), new=_log(rng, 16, 2048), past=rng.choice((0, 0, _log(rng, 1, 4096))))
    # a bound on the cache that one case holds: 64 sequences of 8 K tokens with 8 heads of 128
    c["past"] = min(c["past"], 64 * 8192 * 8 * 128 // (c["b"] * hkv * d))
    if op == "append":
        c.update(rot=rng.choice((d, d, d // 2, d // 4)), inter=rng.random() < 0.4)
    return c


def _lens(case):
    """(new tokens, tokens in the cache with them) of every sequence: the first has the
    case's largest counts, the others any smaller ones, an idle sequence now and then
    where more than one token may come."""
    rng = random.Random(case["mix"])
    new, ctx = [], []
    for b in range(case["b"]):
        n = case["new"] if b == 0 or case["new"] == 1 else rng.randrange(0, case["new"] + 1)
        past = case["past"] if b == 0 else rng.randrange(0, case["past"] + 1)
        new.append(n)
        ctx.append(past + n)
    return new, ctx


SCALING = {"none": {}, "linear": {"factor": 4.0},
           "bands": {"factor": 8.0, "low": 1.0, "high": 4.0, "trained": 8192},
           "yarn": {"factor": 16.0, "low": 1.0, "high": 32.0, "trained": 4096}}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _scale_of(amax):
    """The power of two 2^e with the least e >= -64 for which amax <= 448 * 2^e."""
    f, x = torch.frexp(amax)
    e = torch.where(f <= 0.875, x - 9, x - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -64)).clamp(min=-64)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _table(positions, rot, base):
    p = torch.arange(positions, device=DEV, dtype=torch.float64)
    f = base ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    a = p[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float()


def prepare(case, seed):
    if case["op"] == "table":
        # a table has no inputs but its parameters: the base moves with the seed
        return {"case": case, "base": case["base"] * (1.0 + (seed % 97) / 1000.0)}
    g = _gen(seed)
    dt, page, hkv, d = TYPES[case["dtype"]], case["page"], case["hkv"], case["d"]
    new, ctx = _lens(case)
    b, rows = case["b"], sum(new)
    t = rows + case["pad"]
    need = [max(1, -(-c // page)) for c in ctx]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=_gen(seed + 1), device=DEV).to(torch.int32)
    table = torch.zeros(b, max(need), dtype=torch.int32)
    host = order.cpu()
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = host[at:at + n]
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s = {"case": case, "rows": rows, "max_q": max(new),
         "cu_q": None if case["new"] == 1 and case["pad"] == 0 else torch.tensor(cu, dtype=torch.int32, device=DEV),
         "ctx": torch.tensor(ctx, dtype=torch.int32, device=DEV), "block_table": table.to(DEV)}
    # keys have a few channels far larger than the others, values do not; the sizes of
    # tokens differ, so the pages' scales do too
    loud = 1.0 + 7.0 * (torch.rand(hkv, 1, d, generator=g, device=DEV) < 0.04)
    size = torch.exp(0.5 * _randn(g, n_pages, hkv, 1, 1))
    k = _randn(g, n_pages, hkv, page, d) * loud * size
    v = _randn(g, n_pages, hkv, d, page) * size
    s["k_scale"] = _scale_of(k.abs().amax((2, 3)))
    s["v_scale"] = _scale_of(v.abs().amax((2, 3)))
    s["k_cache"] = (k / s["k_scale"][:, :, None, None]).to(FP8)
    s["v_cache"] = (v / s["v_scale"][:, :, None, None]).to(FP8)
    del k, v
    if case["op"] == "attn":
        q = _randn(g, t, case["hq"], d) * torch.exp(0.3 * _randn(g, t, case["hq"], 1))
        s["q"] = q.to(dt)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(t, case["hq"], device=DEV)
    else:
        # one row of the stacked q, k and v projections per token
        qkv = _randn(g, t, case["hq"] + 2 * hkv, d) * torch.exp(0.5 * _randn(g, t, 1, 1))
        qkv[:, case["hq"]:case["hq"] + hkv] *= loud[:, 0]
        s["qkv"] = qkv.to(dt)
        s["rope"] = _table(max(ctx) + 5, case["rot"], 500000.0)
        s["q_out"] = torch.zeros(t, case["hq"], d, dtype=dt, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms

def _plain_table(case, base):
    r, sc = case["rot"], SCALING[case["scaling"]]
    j = torch.arange(0, r, 2, device=DEV, dtype=torch.float64)
    f = base ** (-j / r)
    m = 1.0
    if case["scaling"] == "linear":
        f = f / sc["factor"]
    elif case["scaling"] == "bands":
        turns = sc["trained"] * f / (2 * math.pi)
        w = ((turns - sc["low"]) / (sc["high"] - sc["low"])).clamp(0, 1)
        f = w * f + (1 - w) * f / sc["factor"]
    elif case["scaling"] == "yarn":
        def dim(turns):
            return r * math.log(sc["trained"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(dim(sc["high"])), 0), min(math.ceil(dim(sc["low"])), r - 1)
        w = 1 - ((j / 2 - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = w * f + (1 - w) * f / sc["factor"]
        m = 0.1 * math.log(sc["factor"]) + 1.0
    a = torch.arange(case["positions"], device=DEV, dtype=torch.float64)[:, None] * f
    return (torch.cat((a.cos(), a.sin()), 1) * m).float()


def _rows(s):
    """Sequence and position of every new row, first new position of every sequence."""
    b, rows = s["ctx"].numel(), s["rows"]
    cu = s["cu_q"] if s["cu_q"] is not None else torch.arange(b + 1, device=DEV, dtype=torch.int32)
    cu = cu.long()
    r = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), r, right=True)
    first = s["ctx"].long() - (cu[1:] - cu[:-1])
    return cu, seq, first, first[seq] + r - cu[seq]


def _rotate(x, cs, rot, inter):
    c, n = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    y = x.clone()
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * n, b * c + a * n
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * n, b * c + a * n
    return y


def _plain_append(s):
    c = s["case"]
    hq, hkv, page, rows = c["hq"], c["hkv"], c["page"], s["rows"]
    cu, seq, first, pos = _rows(s)
    x = s["qkv"][:rows].float()
    cs = s["rope"][pos]
    s["q_out"][:rows] = _rotate(x[:, :hq], cs, c["rot"], c["inter"]).to(s["q_out"].dtype)
    k, v = _rotate(x[:, hq:hq + hkv], cs, c["rot"], c["inter"]), x[:, hq + hkv:]
    bt = s["block_table"].long()
    at, off = bt[seq, pos // page], pos % page
    # the one page of a sequence that may hold older tokens, and how many
    head = bt[torch.arange(len(bt), device=DEV), (first // page).clamp(max=bt.shape[1] - 1)]
    kept = torch.where(cu[1:] > cu[:-1], first % page, torch.full_like(first, page))
    for x, cache, scale, slot in ((k, s["k_cache"], s["k_scale"], 2), (v, s["v_cache"], s["v_scale"], 3)):
        codes, old = cache.view(torch.uint8), scale.clone()
        amax = torch.zeros_like(scale).index_reduce_(0, at, x.abs().amax(2), "amax")
        made = _scale_of(amax)
        made[head] = torch.where((kept > 0)[:, None], torch.maximum(old[head], made[head]), made[head])
        scale[at] = made[at]
        ratio = (old[head] / scale[head])[:, :, None, None]
        before = codes[head]
        again = (before.view(FP8).float() * ratio).to(FP8).view(torch.uint8)
        i = torch.arange(page, device=DEV)
        i = i[:, None] if slot == 2 else i
        moved = (i < kept[:, None, None, None]) & (cu[1:] > cu[:-1])[:, None, None, None]
        codes[head] = torch.where(moved, again, before)
        new = (x / scale[at][:, :, None]).to(FP8).view(torch.uint8)
        if slot == 2:
            codes[at, :, off] = new
        else:
            codes[at, :, :, off] = new


def _plain_attn(s):
    c = s["case"]
    hq, hkv, d, page, rows, mq = c["hq"], c["hkv"], c["d"], c["page"], s["rows"], s["max_q"]
    if not rows:
        return
    cu, seq, first, pos = _rows(s)
    bt = s["block_table"].long()
    b, n = len(bt), bt.shape[1] * page
    k = s["k_cache"][bt].float() * s["k_scale"][bt][..., None, None]
    k = k.permute(0, 2, 1, 3, 4).reshape(b, hkv, n, d)
    v = s["v_cache"][bt].float() * s["v_scale"][bt][..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(b, hkv, n, d)
    i = torch.arange(mq, device=DEV)
    q = s["q"].float()[(cu[:-1, None] + i).clamp(max=rows - 1)]                    # [b, mq, hq, d]
    q = q.view(b, mq, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    x = torch.matmul(q, k.transpose(2, 3)).view(b, hkv, mq, hq // hkv, n).mul_(d ** -0.5)
    unseen = torch.arange(n, device=DEV) > (first[:, None] + i)[:, :, None]
    x.masked_fill_(unseen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(b, hkv, -1, n), v).view(b, hkv, mq, -1, d) / total.clamp(min=1e-30)
    o = o.permute(0, 2, 1, 3, 4).reshape(b, mq, hq, d)
    lse = (top + total.log()).squeeze(-1).permute(0, 2, 1, 3).reshape(b, mq, hq)
    at = torch.arange(rows, device=DEV) - cu[seq]
    s["out"][:rows] = o[seq, at].to(s["out"].dtype)
    s["lse"][:rows] = lse[seq, at]


def run(s):
    c = s["case"]
    if own:
        import weight_only_int4_awq_amd as P
    if c["op"] == "table":
        if not own:
            return _plain_table(c, s["base"])
        sc = SCALING[c["scaling"]]
        return P.awq_rope_table(c["positions"], c["rot"], base=s["base"], scaling=c["scaling"], **sc)
    if c["op"] == "append":
        if own:
            hq, hkv = c["hq"], c["hkv"]
            qkv = s["qkv"]
            fn = P.awq_kv8_append if c["dtype"] == "fp16" else P.awq_kv8_append_bf16
            fn(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
               s["block_table"], s["ctx"], cu_q=s["cu_q"], q=qkv[:, :hq], rope=s["rope"], interleaved=c["inter"],
               out=s["q_out"])
        else:
            _plain_append(s)
        return {n: s[n] for n in ("q_out", "k_cache", "v_cache", "k_scale", "v_scale")}
    if own:
        fn = P.awq_attn_kv8 if c["dtype"] == "fp16" else P.awq_attn_kv8_bf16
        fn(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"], s["ctx"],
           cu_q=s["cu_q"], max_q=s["max_q"], out=s["out"], lse=s["lse"])
    else:
        _plain_attn(s)
    return {"out": s["out"], "lse": s["lse"]}


def work(case):
    if case["op"] == "table":
        n = case["positions"] * case["rot"]
        return {"bytes": 4 * n, "flops": 20 * n}
    new, ctx = _lens(case)
    t, hq, hkv, d, b = sum(new), case["hq"], case["hkv"], case["d"], case["b"]
    if case["op"] == "append":
        return {"bytes": t * (4 * hq * d + 6 * hkv * d + 4 * case["rot"]) + 4 * b,
                "flops": t * (3 * (hq + hkv) * case["rot"] + 4 * hkv * d)}
    live = [c for n, c in zip(new, ctx) if n]
    pairs = sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(new, ctx))
    return {"bytes": 2 * sum(live) * hkv * d + t * (4 * hq * d + 4 * hq), "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------- from the definition, in 64 bits

def _e4m3(x):
    """The nearest e4m3 value (ties to the even code) of |x| <= 448, in float64."""
    e = torch.frexp(x)[1] - 1
    unit = torch.ldexp(torch.ones_like(x), e.clamp(min=-6) - 3)
    return torch.round(x / unit) * unit


def _exact_scale(amax):
    s = torch.full_like(amax, 2.0 ** -64)
    while bool((amax > 448 * s).any()):
        s = torch.where(amax > 448 * s, s * 2, s)
    return s


def _exact_append(s):
    c = s["case"]
    new, ctx = _lens(c)
    hq, hkv, page, rot = c["hq"], c["hkv"], c["page"], c["rot"]
    kc, vc, ks, vs = (s[n].double() for n in ("k_cache", "v_cache", "k_scale", "v_scale"))
    q = s["q_out"].double()
    half = rot // 2
    lo = torch.arange(half, device=DEV) * 2 if c["inter"] else torch.arange(half, device=DEV)
    hi = lo + 1 if c["inter"] else lo + half
    row = 0
    for b, (n, end) in enumerate(zip(new, ctx)):
        if not n:
            continue
        x = s["qkv"][row:row + n].double()
        cs = s["rope"][end - n:end].double()
        turned = x[:, :hq + hkv].clone()
        z = torch.complex(x[:, :hq + hkv][..., lo], x[:, :hq + hkv][..., hi]) \
            * torch.complex(cs[:, :half], cs[:, half:])[:, None]
        turned[..., lo], turned[..., hi] = z.real, z.imag
        q[row:row + n] = turned[:, :hq]
        k, v = turned[:, hq:], x[:, hq + hkv:]
        for j in range((end - n) // page, (end - 1) // page + 1):
            at = int(s["block_table"][b, j])
            a, z = max(end - n, j * page), min(end, (j + 1) * page)
            old = a - j * page
            for y, cache, scale in ((k, kc, ks), (v, vc.transpose(2, 3), vs)):
                part = y[a - end + n:z - end + n].transpose(0, 1)                  # [hkv, new, d]
                m = _exact_scale(part.abs().amax((1, 2)))
                if old:
                    m = torch.maximum(m, scale[at])
                    cache[at, :, :old] = _e4m3(cache[at, :, :old] * (scale[at] / m)[:, None, None])
                cache[at, :, old:z - j * page] = _e4m3(part / m[:, None, None])
                scale[at] = m
        row += n
    return {"q_out": q, "k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs}


def _exact_attn(s):
    c = s["case"]
    new, ctx = _lens(c)
    hkv, g, d = c["hkv"], c["hq"] // c["hkv"], c["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    row = 0
    for b, (n, end) in enumerate(zip(new, ctx)):
        pages = s["block_table"][b, :-(-end // c["page"])].long() if n else None
        for h in range(hkv if n else 0):
            k = (s["k_cache"][pages, h].double() * s["k_scale"][pages, h].double()[:, None, None]).reshape(-1, d)[:end]
            v = (s["v_cache"][pages, h].double() * s["v_scale"][pages, h].double()[:, None, None]) \
                .transpose(1, 2).reshape(-1, d)[:end]
            for r in range(0, n, 1024):
                m = min(1024, n - r)
                last = end - n + r + m                                              # keys that any of them sees
                q = s["q"][row + r:row + r + m, h * g:(h + 1) * g].double()
                x = torch.matmul(q.reshape(-1, d), k[:last].t().contiguous()).view(m, g, last) / math.sqrt(d)
                own_pos = torch.arange(last - m, last, device=DEV)
                x = x.masked_fill((torch.arange(last, device=DEV) > own_pos[:, None])[:, None], -math.inf)
                z = torch.logsumexp(x, -1)
                out[row + r:row + r + m, h * g:(h + 1) * g] = torch.matmul(
                    torch.exp(x - z[..., None]).view(m * g, last), v[:last]).view(m, g, d)
                lse[row + r:row + r + m, h * g:(h + 1) * g] = z
        row += n
    return {"out": out, "lse": lse}


def _exact_table(case, base):
    """From the complex exponential, one factor for each binary digit of the position."""
    r, sc, kind = case["rot"], SCALING[case["scaling"]], case["scaling"]
    freq, m = [], 1.0
    for j in range(r // 2):
        f = math.exp(-2.0 * j / r * math.log(base))
        if kind == "linear":
            f /= sc["factor"]
        elif kind == "bands":
            wave = 2 * math.pi / f
            if wave > sc["trained"] / sc["low"]:
                f /= sc["factor"]
            elif wave >= sc["trained"] / sc["high"]:
                w = (sc["trained"] / wave - sc["low"]) / (sc["high"] - sc["low"])
                f *= w + (1 - w) / sc["factor"]
        elif kind == "yarn":
            first, last = (r / 2 * math.log(sc["trained"] / (2 * math.pi * sc[n]), base) for n in ("high", "low"))
            first, last = max(math.floor(first), 0), min(math.ceil(last), r - 1)
            ramp = min(max((j - first) / max(last - first, 1e-3), 0.0), 1.0)
            f *= 1 - ramp + ramp / sc["factor"]
            m = 1.0 + math.log(sc["factor"]) / 10
        freq.append(f)
    p = torch.arange(case["positions"], device=DEV)
    f = torch.tensor(freq, dtype=torch.float64, device=DEV)
    z = torch.ones(len(p), len(f), dtype=torch.complex128, device=DEV)
    for bit in range(max(1, case["positions"].bit_length())):
        turn = torch.polar(torch.ones_like(f), torch.remainder(f * (1 << bit), 2 * math.pi))
        z = torch.where(((p >> bit) & 1).bool()[:, None], z * turn, z)
    return torch.cat((z.real, z.imag), 1) * m


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "table":
        return _exact_table(case, s["base"])
    return _exact_append(s) if case["op"] == "append" else _exact_attn(s)
