"""Mixture-of-experts layers with packed experts, and linears with a fused epilogue: what is
measured of awq_moe_route, awq_moe_linear_w4a16, awq_moe_combine and awq_linear_w4a16_act,
with their plain forms in elementary torch operations.

A mixture-of-experts block routes each of t tokens to its topk best of e experts (route),
runs the tokens of every expert through that expert's packed gate and up projection and then
its down projection (linear, grouped by expert), and adds the experts' results by their
weights (combine).  The plan between them:

  ids, weights [t][topk]   the experts of a token, best first (-1 and 0 where fewer are open)
  offsets [e + 1]          rows offsets[i] .. offsets[i + 1] - 1 belong to expert i
  row_slot [t * topk]      slot (token * topk + choice) of every row: by expert, then by slot
  slot_row [t][topk]       row of every slot, -1 where it has none

Dense layers end in a bias, an activation (of one projection, or of a gate that multiplies a
second projection) and the addition of a residual (act).

Packed weights: code k of row n in bits 4 (k % 8) .. of qweight[n][k / 8], scales[n][k / g]
fp16, zero point j of row n in bits 4 (j % 8) .. of qzeros[n][j / 8]; the value of a code is
(code - zero point) * scale.  A gated projection has its n gate rows first, then n up rows.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoding token among 8 experts: the smallest call
        {"name": "route_1_of_8", "op": "route", "dtype": "fp32", "t": 1, "e": 8, "topk": 2, "scoring": "softmax",
         "renorm": True, "scale": 1.0, "closed": 0, "pad": 0},
        # a prompt of odd length among 128 experts, five of them closed, padded tokens behind it
        {"name": "route_8k_of_128", "op": "route", "dtype": "bf16", "t": 8191, "e": 128, "topk": 8,
         "scoring": "sigmoid", "renorm": True, "scale": 2.5, "closed": 5, "pad": 100},
        # gate and up projection: one token, two of 8 large experts (weights read once)
        {"name": "experts_1_of_8", "op": "experts", "dtype": "fp16", "t": 1, "e": 8, "topk": 2, "n": 14336, "k": 4096,
         "g": 128, "gated": True, "act": "silu", "bias": False, "inv": False, "gather": True, "pad": 0, "mix": 1},
        # a batch of 64 decoding tokens on 128 small experts: four ragged rows each
        {"name": "experts_64_of_128", "op": "experts", "dtype": "bf16", "t": 64, "e": 128, "topk": 8, "n": 1024,
         "k": 2048, "g": 128, "gated": True, "act": "silu", "bias": False, "inv": False, "gather": True, "pad": 0,
         "mix": 2},
        # the down projection of a batch of short prompts on 60 experts, biases, odd lengths, padded tokens
        {"name": "experts_down_300_of_60", "op": "experts", "dtype": "fp16", "t": 300, "e": 60, "topk": 4, "n": 2048,
         "k": 1408, "g": 64, "gated": False, "act": "none", "bias": True, "inv": False, "gather": False, "pad": 13,
         "mix": 3},
        # gate and up projection of a prompt on 8 large experts (products bound it)
        {"name": "experts_4k_of_8", "op": "experts", "dtype": "fp16", "t": 4096, "e": 8, "topk": 2, "n": 14336,
         "k": 4096, "g": 128, "gated": True, "act": "silu", "bias": False, "inv": False, "gather": True, "pad": 0,
         "mix": 4},
        # the sums of a decoding batch, and of a prompt with the residual stream
        {"name": "combine_64", "op": "combine", "dtype": "bf16", "t": 64, "topk": 8, "n": 2048, "residual": True,
         "pad": 0},
        {"name": "combine_8k", "op": "combine", "dtype": "fp16", "t": 8191, "topk": 8, "n": 4096, "residual": True,
         "pad": 100},
        # a dense layer's gate and up projection for one token
        {"name": "act_gate_up_1", "op": "act", "dtype": "fp16", "m": 1, "n": 14336, "k": 4096, "g": 128, "gated": True,
         "act": "silu", "bias": False, "inv": True, "residual": False},
        # an output projection onto the residual stream, a small decoding batch
        {"name": "act_out_17", "op": "act", "dtype": "bf16", "m": 17, "n": 4096, "k": 4096, "g": 128, "gated": False,
         "act": "none", "bias": False, "inv": True, "residual": True},
        # a projection with bias and gelu, odd widths, a chunk of a prompt
        {"name": "act_bias_gelu_333", "op": "act", "dtype": "fp16", "m": 333, "n": 4099, "k": 1088, "g": 64,
         "gated": False, "act": "gelu", "bias": True, "inv": False, "residual": False},
        # a down projection of a prompt onto the residual stream (products bound it)
        {"name": "act_down_2048", "op": "act", "dtype": "bf16", "m": 2048, "n": 4096, "k": 14336, "g": 128,
         "gated": False, "act": "none", "bias": False, "inv": True, "residual": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "experts", "experts", "experts", "combine", "act", "act", "act"))
    if op == "route":
        e = _log(rng, 2, 256)
        t = _log(rng, 1, 8191)
        return {"op": op, "dtype": rng.choice(("fp32", "fp16", "bf16")), "t": t, "e": e,
                "topk": rng.randrange(1, min(e, 8) + 1), "scoring": rng.choice(("softmax", "sigmoid")),
                "renorm": rng.random() < 0.7, "scale": rng.choice((1.0, 2.5)), "closed": rng.choice((0, 0, e // 3)),
                "pad": rng.choice((0, 0, t // 4))}
    dt = rng.choice(("fp16", "bf16"))
    if op == "combine":
        t = _log(rng, 1, 8191)
        return {"op": op, "dtype": dt, "t": t, "topk": rng.randrange(1, 9), "n": 8 * _log(rng, 32, 512),
                "residual": rng.random() < 0.6, "pad": rng.choice((0, 0, t // 4))}
    g = rng.choice((128, 128, 128, 64, 32))
    k = max(g, 64) * _log(rng, 1, 4096 // max(g, 64))
    n = rng.choice((_log(rng, 40, 8192), 64 * _log(rng, 1, 128)))
    act = rng.choice(("none", "silu", "gelu", "gelu_tanh"))
    c = {"op": op, "dtype": dt, "n": n, "k": k, "g": g, "act": act, "gated": act != "none" and rng.random() < 0.6,
         "bias": rng.random() < 0.3, "inv": rng.random() < 0.4}
    if op == "act":
        c.update(m=_log(rng, 1, 4096), residual=rng.random() < 0.5)
        return c
    e = _log(rng, 2, 128)
    c["n"] = max(16, min(n, 128 * 2048 * 2048 // (e * k)))            # a bound on the experts' weights
    c.update(t=_log(rng, 1, 4096), e=e, topk=rng.randrange(1, min(e, 8) + 1), gather=rng.random() < 0.6,
             pad=0, mix=rng.randrange(1 << 20))
    c["t"] = min(c["t"], max(1, 9 * 10 ** 11 // (c["n"] * (2 if c["gated"] else 1) * k * c["topk"])))    # and on the work
    c["pad"] = rng.choice((0, 0, c["t"] // 4))
    return c


def _routing(case):
    """Rows of every expert and the slot of every row: some experts are more popular than
    others; the last `pad` tokens have none."""
    gen = torch.Generator().manual_seed(case["mix"])
    t, e, topk = case["t"], case["e"], case["topk"]
    x = 0.7 * torch.randn(e, generator=gen) - torch.log(-torch.log(torch.rand(t, e, generator=gen).clamp(1e-9, 1 - 1e-6)))
    ids = x.topk(topk, 1).indices
    if case["pad"]:
        ids[t - case["pad"]:] = e
    flat = ids.flatten()
    count = torch.bincount(flat, minlength=e + 1)[:e]
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64), count.cumsum(0)))
    return offsets, torch.sort(flat, stable=True).indices


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _tokens(g, rows, k):
    """Activations behind a norm: one channel in a hundred is twenty times as loud."""
    x = _randn(g, rows, k)
    return x * (1.0 + 19.0 * (torch.rand(k, generator=g, device=DEV) < 0.01))


def _packed(g, lead, n, k, group):
    """Packed weights: codes about the middle of their range, zero points next to it."""
    def word(mask, *shape):
        hi = torch.randint(0, 1 << 16, shape, generator=g, device=DEV, dtype=torch.int32)
        lo = torch.randint(0, 1 << 16, shape, generator=g, device=DEV, dtype=torch.int32)
        return ((hi << 16) | lo) & mask
    shape = (*lead, n, k // 8)
    qw = word(0x77777777, *shape) + word(0x77777777, *shape) + word(0x11111111, *shape)    # every field stays below 16
    ng = k // group
    sc = (0.0055 * torch.exp(0.2 * _randn(g, *lead, n, ng))).half()
    fields = word(0x11111111, *lead, n, -(-ng // 8)) + word(0x11111111, *lead, n, -(-ng // 8)) + 0x66666666
    if ng % 8:
        fields[..., -1] &= (1 << (4 * (ng % 8))) - 1
    return qw, sc, fields


def prepare(case, seed):
    g = _gen(seed)
    dt = TYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "route":
        t, e, topk = case["t"], case["e"], case["topk"]
        x = 1.5 * _randn(g, t, e) + 0.7 * _randn(g, e)
        if case["closed"]:
            x[:, torch.randperm(e, generator=g, device=DEV)[:case["closed"]]] = -math.inf
        if case["pad"]:
            x[t - case["pad"]:] = -math.inf
        i32 = {"dtype": torch.int32, "device": DEV}
        s["logits"] = x.to(dt)
        s["out"] = (torch.zeros(t, topk, **i32), torch.zeros(t, topk, device=DEV), torch.zeros(e + 1, **i32),
                    torch.zeros(t * topk, **i32), torch.zeros(t, topk, **i32))
        return s
    if case["op"] == "combine":
        t, topk = case["t"], case["topk"]
        s["rows"] = _randn(g, t * topk, case["n"]).to(dt)
        s["weights"] = torch.softmax(_randn(g, t, topk), 1)
        slot_row = torch.randperm(t * topk, generator=g, device=DEV).view(t, topk)
        if case["pad"]:
            slot_row[t - case["pad"]:] = -1
            s["weights"][t - case["pad"]:] = 0
        s["slot_row"] = slot_row.to(torch.int32)
        s["residual"] = (3.0 * _randn(g, t, case["n"])).to(dt) if case["residual"] else None
        s["out"] = torch.zeros(t, case["n"], dtype=dt, device=DEV)
        return s
    n, k, act = case["n"], case["k"], case["op"] == "act"
    wide = 2 * n if case["gated"] else n
    lead = () if act else (case["e"],)
    s["w"] = _packed(g, lead, wide, k, case["g"])
    s["bias"] = (0.5 * _randn(g, *lead, wide)).to(dt) if case["bias"] else None
    s["inv"] = torch.exp(0.3 * _randn(g, k)).half() if case["inv"] else None
    if act:
        s["x"] = _tokens(g, case["m"], k).to(dt)
        s["residual"] = (3.0 * _randn(g, case["m"], n)).to(dt) if case["residual"] else None
        s["out"] = torch.zeros(case["m"], n, dtype=dt, device=DEV)
    else:
        offsets, row_slot = _routing(case)
        rows = case["t"] * case["topk"]
        s["offsets"], s["row_slot"] = offsets.to(DEV, torch.int32), row_slot.to(DEV, torch.int32)
        s["x"] = _tokens(g, case["t"] if case["gather"] else rows, k).to(dt)
        s["out"] = torch.zeros(rows, n, dtype=dt, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms

def _plain_route(s):
    c = s["case"]
    e, topk = c["e"], c["topk"]
    x = s["logits"].float()
    best, ids = torch.sort(x, dim=1, descending=True, stable=True)
    best, ids = best[:, :topk], ids[:, :topk]
    open_ = best > -math.inf
    if c["scoring"] == "softmax":
        top = torch.where(open_[:, :1], best[:, :1], torch.zeros_like(best[:, :1]))
        w = torch.exp(best - top)
        if not c["renorm"]:
            w = w / torch.exp(x - top).sum(1, keepdim=True).clamp(min=1e-30)
    else:
        w = 1.0 / (1.0 + torch.exp(-best))
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    w = torch.where(open_, w * c["scale"], torch.zeros_like(w))
    flat = torch.where(open_, ids, torch.full_like(ids, e)).flatten()
    order = torch.sort(flat, stable=True).indices
    count = torch.zeros(e + 1, dtype=torch.int64, device=DEV).index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64, device=DEV), count[:e].cumsum(0)))
    at = torch.arange(len(flat), device=DEV)
    used = at < offsets[e]
    slot_row = torch.empty_like(order)
    slot_row[order] = torch.where(used, at, torch.full_like(at, -1))
    return {"ids": torch.where(open_, ids, torch.full_like(ids, -1)).int(), "weights": w, "offsets": offsets.int(),
            "row_slot": torch.where(used, order, s["out"][3].long()).int(), "slot_row": slot_row.view(-1, topk).int()}


def _unpack(words, count):
    """The first `count` 4-bit fields of every row of words, lowest first."""
    f = torch.stack([(words >> (4 * i)) & 15 for i in range(8)], -1)
    return f.flatten(-2)[..., :count]


def _weight(w, g):
    qw, sc, qz = w
    k, ng = qw.shape[-1] * 8, sc.shape[-1]
    q = _unpack(qw, k).view(*qw.shape[:-1], ng, g) - _unpack(qz, ng)[..., None]
    return (q.float() * sc.float()[..., None]).view(*qw.shape[:-1], k)


def _activate(x, kind):
    if kind == "silu":
        return x / (1.0 + torch.exp(-x))
    if kind == "gelu":
        return 0.5 * x * torch.special.erfc(x * -math.sqrt(0.5))
    if kind == "gelu_tanh":
        return x / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _plain_linear(x, w, bias, case):
    y = torch.matmul(x, _weight(w, case["g"]).t())
    if bias is not None:
        y += bias.float()
    if not case["gated"]:
        return _activate(y, case["act"])
    n = case["n"]
    return _activate(y[:, :n], case["act"]) * y[:, n:]


def _plain_experts(s):
    c = s["case"]
    out = s["out"]
    x = s["x"].float()
    if s["inv"] is not None:
        x = x * s["inv"].float()
    at = s["offsets"].tolist()
    for i in range(c["e"]):
        a, z = at[i], at[i + 1]
        if a < z:
            rows = s["row_slot"][a:z].long() // c["topk"] if c["gather"] else torch.arange(a, z, device=DEV)
            y = _plain_linear(x[rows], [p[i] for p in s["w"]], None if s["bias"] is None else s["bias"][i], c)
            out[a:z] = y.to(out.dtype)
    return out


def _plain_act(s):
    c = s["case"]
    x = s["x"].float()
    if s["inv"] is not None:
        x = x * s["inv"].float()
    y = _plain_linear(x, s["w"], s["bias"], c)
    if s["residual"] is not None:
        y += s["residual"].float()
    return y.to(s["out"].dtype)


def _plain_combine(s):
    rows = s["slot_row"].long()
    y = s["residual"].float() if s["residual"] is not None else torch.zeros(s["out"].shape, device=DEV)
    for j in range(rows.shape[1]):
        r = rows[:, j]
        part = s["rows"][r.clamp(min=0)].float() * s["weights"][:, j, None]
        y = y + torch.where((r >= 0)[:, None], part, torch.zeros_like(part))
    return y.to(s["out"].dtype)


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "route":
            return _plain_route(s)
        return {"y": {"experts": _plain_experts, "act": _plain_act, "combine": _plain_combine}[op](s)}
    import weight_only_int4_awq_amd as P
    if op == "route":
        out = P.awq_moe_route(s["logits"], c["topk"], scoring=c["scoring"], renormalize=c["renorm"], scale=c["scale"],
                              out=s["out"])
        return dict(zip(("ids", "weights", "offsets", "row_slot", "slot_row"), out))
    fp16 = c["dtype"] == "fp16"
    if op == "combine":
        fn = P.awq_moe_combine if fp16 else P.awq_moe_combine_bf16
        return {"y": fn(s["rows"], s["weights"], s["slot_row"], residual=s["residual"], out=s["out"])}
    if op == "act":
        fn = P.awq_linear_w4a16_act if fp16 else P.awq_linear_w4a16_act_bf16
        return {"y": fn(s["x"], *s["w"], inv_s16=s["inv"], bias=s["bias"], act=c["act"], gated=c["gated"],
                        residual=s["residual"], g=c["g"], out=s["out"])}
    fn = P.awq_moe_linear_w4a16 if fp16 else P.awq_moe_linear_w4a16_bf16
    return {"y": fn(s["x"], *s["w"], s["offsets"], row_slot=s["row_slot"] if c["gather"] else None, topk=c["topk"],
                    inv_s16=s["inv"], bias=s["bias"], act=c["act"], gated=c["gated"], g=c["g"], out=s["out"])}


def work(case):
    op = case["op"]
    if op == "route":
        t, e, topk = case["t"], case["e"], case["topk"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": t * e * size + 16 * t * topk + 4 * (e + 1), "flops": t * e * 4}
    n = case["n"]
    if op == "combine":
        t, topk = case["t"], case["topk"]
        used = (t - case["pad"]) * topk
        return {"bytes": 2 * n * (used + t + (t if case["residual"] else 0)) + 8 * t * topk, "flops": 2 * n * used}
    k, ng = case["k"], case["k"] // case["g"]
    wide = 2 * n if case["gated"] else n
    each = wide * (k // 2 + 2 * ng + 4 * (-(-ng // 8)) + (2 if case["bias"] else 0))
    inv = 2 * k if case["inv"] else 0
    if op == "act":
        m = case["m"]
        return {"bytes": each + inv + 2 * m * (k + n + (n if case["residual"] else 0)), "flops": 2 * m * wide * k}
    offsets, _ = _routing(case)
    rows, live = int(offsets[-1]), int((offsets[1:] > offsets[:-1]).sum())
    x = 2 * k * min(rows, case["t"] - case["pad"]) if case["gather"] else 2 * k * rows
    return {"bytes": live * each + inv + x + 2 * rows * n + 4 * (case["e"] + 1) + (4 * rows if case["gather"] else 0),
            "flops": 2 * rows * wide * k}


# ---------------------------------------------------------------- from the definition, in 64 bits

def _exact_route(s):
    """One token at a time, on the host."""
    c = s["case"]
    e, topk = c["e"], c["topk"]
    t = c["t"]
    ids, weights = torch.full((t, topk), -1, dtype=torch.int32), torch.zeros(t, topk, dtype=torch.float64)
    lists = [[] for _ in range(e)]
    for i, row in enumerate(s["logits"].double().tolist()):
        order = sorted((j for j in range(e) if row[j] > -math.inf), key=lambda j: (-row[j], j))
        if not order:
            continue
        if c["scoring"] == "softmax":
            p = {j: math.exp(row[j] - row[order[0]]) for j in order}
            total = math.fsum(p.values())
            p = {j: p[j] / total for j in order}
        else:
            p = {j: 0.5 * (1.0 + math.tanh(row[j] / 2)) if row[j] > -1 else math.exp(row[j]) / (1 + math.exp(row[j]))
                 for j in order}
        order = order[:topk]
        total = math.fsum(p[j] for j in order) if c["renorm"] else 1.0
        for a, j in enumerate(order):
            ids[i, a] = j
            weights[i, a] = p[j] / total * c["scale"]
            lists[j].append(i * topk + a)
    offsets, row_slot = [0], s["out"][3].cpu()
    slot_row = torch.full((t * topk,), -1, dtype=torch.int32)
    for slots in lists:
        for r, slot in enumerate(slots, offsets[-1]):
            row_slot[r] = slot
            slot_row[slot] = r
        offsets.append(offsets[-1] + len(slots))
    made = {"ids": ids, "weights": weights, "offsets": torch.tensor(offsets, dtype=torch.int32), "row_slot": row_slot,
            "slot_row": slot_row.view(t, topk)}
    return {n: v.to(DEV) for n, v in made.items()}


def _exact_weight(w, g):
    """From bytes: a byte holds two codes, the even one low."""
    qw, sc, qz = w
    n, ng = sc.shape
    b = qw.contiguous().view(torch.uint8).view(n, -1)
    q = torch.empty(n, b.shape[1] * 2, dtype=torch.float64, device=DEV)
    q[:, 0::2], q[:, 1::2] = (b % 16).double(), (b // 16).double()
    b = qz.contiguous().view(torch.uint8).view(n, -1)
    z = torch.empty(n, b.shape[1] * 2, dtype=torch.float64, device=DEV)
    z[:, 0::2], z[:, 1::2] = (b % 16).double(), (b // 16).double()
    q -= z[:, :ng].repeat_interleave(g, 1)
    return q * sc.double().repeat_interleave(g, 1)


def _exact_linear(x, w, bias, case):
    n, kind = case["n"], case["act"]
    full = _exact_weight(w, case["g"])
    parts = []
    for part in range(2 if case["gated"] else 1):
        y = torch.matmul(x, full[part * n:(part + 1) * n].t().contiguous())
        parts.append(y if bias is None else y + bias[part * n:(part + 1) * n].double())
    y = parts[0]
    if kind == "silu":
        y = y * torch.sigmoid(y)
    elif kind == "gelu":
        y = y * 0.5 * torch.special.erfc(-y / math.sqrt(2.0))
    elif kind == "gelu_tanh":
        y = y * torch.sigmoid(math.sqrt(8.0 / math.pi) * (y + 0.044715 * y ** 3))
    return y * parts[1] if case["gated"] else y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "combine":
        r = s["slot_row"].long()
        y = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        for j in range(case["topk"]):
            on = (r[:, j] >= 0).nonzero().flatten()
            y[on] += s["weights"][on, j].double()[:, None] * s["rows"][r[on, j]].double()
        return {"y": y if s["residual"] is None else y + s["residual"].double()}
    x = s["x"].double()
    if s["inv"] is not None:
        x = x * s["inv"].double()
    if op == "act":
        y = _exact_linear(x, s["w"], s["bias"], case)
        return {"y": y if s["residual"] is None else y + s["residual"].double()}
    y = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    ends = s["offsets"].tolist()
    token = torch.div(s["row_slot"].long(), case["topk"], rounding_mode="floor")
    for i in range(case["e"]):
        rows = torch.arange(ends[i], ends[i + 1], device=DEV)
        if len(rows):
            y[rows] = _exact_linear(x[token[rows]] if case["gather"] else x[rows], [p[i] for p in s["w"]],
                                    None if s["bias"] is None else s["bias"][i], case)
    return {"y": y}
