"""Float64 reference of the linears with an epilogue, of routing, of products grouped by expert
and of the combination, with bounds on the kernels' results derived from their arithmetic.

A linear's sum before the activation, v = sum_k x~ w:
  * x~ = fp16(x inv_s): 2^-11 relative, 2^-25 absolute (subnormals); exact without inv_s (x is fp16,
    or bf16 within fp16's normal range);
  * w = fp16((q - z) D): 2^-11 relative, 2^-25 absolute; or exact (then the bound is slack);
  * products of two fp16 values are exact in fp32; sums of k of them in fp32, whatever the order:
    k 2^-24 relative of the sum of magnitudes (and 8 roundings more for scales and joins).
The activations grow by at most 1.13 per unit (silu 1.0998, gelu and its tanh form 1.1290); they
are off by 4e-6 relative (exponentials and reciprocals within 2 units of 2^-23 of a value whose
argument is rounded: 16 2^-23 covers |argument| up to 12, beyond which the result is below 1e-5
of its argument).  The result is rounded once: half a unit, 2^-25 where fp16 is subnormal.
"""
from __future__ import annotations

import math

import torch

ACTS = ("none", "silu", "gelu", "gelu_tanh")
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def unpack(words, count):
    f = torch.stack([(words.long() >> (4 * i)) & 15 for i in range(8)], -1)
    return f.flatten(-2)[..., :count]


def weights(qw, sc, qz, g):
    k, ng = qw.shape[-1] * 8, sc.shape[-1]
    q = unpack(qw, k).view(*qw.shape[:-1], ng, g) - unpack(qz, ng)[..., None]
    return (q.double() * sc.double()[..., None]).view(*qw.shape[:-1], k)


def packed(gen, lead, n, k, g, scale=0.02):
    """Random packed weights in layout v1; unused zero fields are 0."""
    ng = k // g
    def bits(*shape):
        return torch.randint(-2 ** 31, 2 ** 31, shape, generator=gen, dtype=torch.int64).to(torch.int32)
    sc = (scale * torch.exp(0.5 * torch.randn(*lead, n, ng, generator=gen))).half()
    qz = bits(*lead, n, -(-ng // 8))
    if ng % 8:
        qz[..., -1] &= (1 << (4 * (ng % 8))) - 1
    return bits(*lead, n, k // 8), sc, qz


def activate(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2.0))
    if act == "gelu_tanh":
        return v * torch.sigmoid(math.sqrt(8.0 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def linear(x, w, inv, bias, act, gated, residual, dtype):
    """(value, bound) of a linear with its epilogue on CPU tensors (w: float64 [nw, k])."""
    x = x.double()
    k = x.shape[1]
    ea, xs = 0.0, x
    if inv is not None:
        xs, ea = x * inv.double(), 2.0 ** -11
    v = xs @ w.t()
    mag = xs.abs() @ w.abs().t()
    gamma = (k + 8) * 2.0 ** -24
    dv = (ea + 2.0 ** -11 + gamma) * 1.01 * mag + 2.0 ** -25 * (xs.abs().sum(1, keepdim=True) + w.abs().sum(1)[None])
    if bias is not None:
        v = v + bias.double()
        dv = dv + 2.0 ** -23 * v.abs()
    n = w.shape[0] // 2 if gated else w.shape[0]

    a, da = activate(v[:, :n], act), dv[:, :n]
    if act != "none":
        da = 1.13 * da + 4e-6 * a.abs()
    if gated:
        u, du = v[:, n:], dv[:, n:]
        a, da = a * u, u.abs() * da + a.abs() * du + da * du + 2.0 ** -22 * (a * u).abs()
    if residual is not None:
        a = a + residual.double()
        da = da + 2.0 ** -23 * (a.abs() + residual.double().abs())
    return a, da + HALF[dtype] * 1.01 * (a.abs() + da) + (2.0 ** -25 if dtype is torch.float16 else 1e-40)


def check(got, value, bound, what=""):
    err = (got.double().cpu() - value).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((err / bound).nan_to_num(1e9).max()),
                           [int(i) for i in bad.nonzero()[0]])


def route(logits, topk, scoring, renormalize, scale):
    """One token at a time.  Rows behind the last are -7 in row_slot."""
    x = logits.double()
    t, e = x.shape
    ids, w = torch.full((t, topk), -1, dtype=torch.int32), torch.zeros(t, topk, dtype=torch.float64)
    lists = [[] for _ in range(e)]
    for i, row in enumerate(x.tolist()):
        order = sorted((j for j in range(e) if row[j] == row[j] and row[j] > -math.inf), key=lambda j: (-row[j], j))
        if order and scoring == "softmax":
            p = {j: math.exp(row[j] - row[order[0]]) if row[order[0]] < math.inf else math.nan for j in order}
            total = math.fsum(p.values())
            p = {j: v / total for j, v in p.items()}
        else:
            p = {j: 1 / (1 + math.exp(-row[j])) if row[j] > -80 else math.exp(row[j]) for j in order}
        order = order[:topk]
        total = math.fsum(p[j] for j in order) if renormalize else 1.0
        for a, j in enumerate(order):
            ids[i, a], w[i, a] = j, p[j] / total * scale
            lists[j].append(i * topk + a)
        if any(v != v for v in row):
            w[i] = math.nan
    offsets, row_slot, slot_row = [0], torch.full((t * topk,), -7, dtype=torch.int32), torch.full((t * topk,), -1, dtype=torch.int32)
    for slots in lists:
        for r, s in enumerate(slots, offsets[-1]):
            row_slot[r], slot_row[s] = s, r
        offsets.append(offsets[-1] + len(slots))
    return ids, w, torch.tensor(offsets, dtype=torch.int32), row_slot, slot_row.view(t, topk)
