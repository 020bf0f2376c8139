"""The 8-bit paged KV cache on the GPU against its definition (tests/kv8_ref.py): the
cache bit for bit, attention within bounds derived from its arithmetic."""
from __future__ import annotations

import numpy as np
import pytest

import synthetic as S
from oracle import awq_oracle as O
from tests import kv8_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
F8 = torch.float8_e4m3fn
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def P():
    import weight_only_int4_awq_amd as P
    P.load()
    assert torch.cuda.is_available()
    return P


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Case:
    """A batch: lengths, a cache with garbage in every slot that holds no token, and its host copy."""

    def __init__(self, seed, dt, new, ctx, hq, hkv, d, page, pad=0, extra=3, fill=True):
        self.rng = rng = np.random.default_rng(seed)
        self.dt, self.hq, self.hkv, self.d, self.page = dt, hq, hkv, d, page
        self.new, self.ctx = list(new), np.array(ctx, np.int32)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.used = int(self.cu[-1])
        self.rows = self.used + pad
        need = [max(1, -(-int(c) // page)) for c in ctx]
        self.pages = sum(need) + extra
        order = rng.permutation(self.pages)
        # entries behind a sequence's pages are rubbish that nothing may follow
        self.bt = rng.integers(-2 ** 31, 2 ** 31 - 1, (len(ctx), max(need)), dtype=np.int32)
        at = 0
        for i, n in enumerate(need):
            self.bt[i, :n] = order[at:at + n]
            at += n
        # the codes of slots without a token are any, NaN codes among them
        self.kc = rng.integers(0, 256, (self.pages, hkv, page, d), dtype=np.uint8)
        self.vc = rng.integers(0, 256, (self.pages, hkv, d, page), dtype=np.uint8)
        self.ks = (2.0 ** rng.integers(-9, -4, (self.pages, hkv))).astype(np.float32)
        self.vs = (2.0 ** rng.integers(-9, -4, (self.pages, hkv))).astype(np.float32)
        if fill:
            for b, c in enumerate(ctx):
                self.tokens(b, 0, int(c))

    def tokens(self, b, lo, hi):
        """Finite codes in the slots lo .. hi - 1 of sequence b."""
        for j in range(lo // self.page, -(-hi // self.page)):
            a, z = max(lo - j * self.page, 0), min(hi - j * self.page, self.page)
            at = self.bt[b, j]
            x = self.rng.standard_normal((self.hkv, z - a, self.d)) * 60
            y = self.rng.standard_normal((self.hkv, self.d, z - a)) * 60
            self.kc[at, :, a:z] = R.encode(np.clip(x, -448, 448))
            self.vc[at, :, :, a:z] = R.encode(np.clip(y, -448, 448))

    def act(self, heads, size=1.0):
        x = self.rng.standard_normal((self.rows, heads, self.d)) * size
        return torch.from_numpy(x).to(DT[self.dt])

    def upload(self):
        self.dk, self.dv = dev(self.kc).view(F8), dev(self.vc).view(F8)
        self.dks, self.dvs = dev(self.ks), dev(self.vs)
        self.dbt, self.dctx, self.dcu = dev(self.bt), dev(self.ctx), dev(self.cu)
        return self.dk, self.dv, self.dks, self.dvs, self.dbt, self.dctx

    def cache(self):
        return (self.dk.view(torch.uint8).cpu().numpy(), self.dv.view(torch.uint8).cpu().numpy(),
                self.dks.cpu().numpy(), self.dvs.cpu().numpy())


def append_fn(P, dt):
    return P.awq_kv8_append if dt == "fp16" else P.awq_kv8_append_bf16


def attn_fn(P, dt):
    return P.awq_attn_kv8 if dt == "fp16" else P.awq_attn_kv8_bf16


def same_cache(c, want):
    for got, ref, name in zip(c.cache(), want, ("k codes", "v codes", "k_scale", "v_scale")):
        g, r = (got.view(np.uint32), ref.view(np.uint32)) if got.dtype == np.float32 else (got, ref)
        assert np.array_equal(g, r), (name, int((g != r).sum()), np.argwhere(g != r)[:4].tolist())


# ---------------------------------------------------------------- rotary table

@pytest.mark.parametrize("positions,rot,base,scaling,kw", [
    (1, 2, 10000.0, "none", {}), (300, 128, 500000.0, "none", {}), (4097, 96, 10000.0, "linear", {"factor": 4.0}),
    (1000003, 16, 10000.0, "none", {}),
    (9000, 128, 500000.0, "bands", {"factor": 8.0, "low": 1.0, "high": 4.0, "trained": 8192}),
    (5000, 64, 10000.0, "yarn", {"factor": 16.0, "low": 1.0, "high": 32.0, "trained": 4096}),
    (77, 256, 10000.0, "yarn", {"factor": 2.5, "low": 2.0, "high": 3.0, "trained": 100})])
def test_rope_table(P, positions, rot, base, scaling, kw):
    got = P.awq_rope_table(positions, rot, base=base, scaling=scaling, **kw).cpu().numpy().astype(np.float64)
    j = np.arange(rot // 2)
    f = base ** (-2.0 * j / rot)
    m = 1.0
    if scaling == "linear":
        f = f / kw["factor"]
    elif scaling == "bands":
        w = np.clip((kw["trained"] * f / (2 * np.pi) - kw["low"]) / (kw["high"] - kw["low"]), 0, 1)
        f = w * f + (1 - w) * f / kw["factor"]
    elif scaling == "yarn":
        def n(t):
            return rot * np.log(kw["trained"] / (2 * np.pi * t)) / (2 * np.log(base))
        lo, hi = max(np.floor(n(kw["high"])), 0), min(np.ceil(n(kw["low"])), rot - 1)
        w = np.clip((j - lo) / max(hi - lo, 0.001), 0, 1)
        f = (1 - w) * f + w * f / kw["factor"]
        m = 0.1 * np.log(kw["factor"]) + 1
    a = np.arange(positions)[:, None] * f
    # 2 ulp of m in fp32 (2 * 2^-23 m), and float64 angles of 10^6 off by 2^-33
    tol = m * (2.0 ** -22 + 2.0 ** -32)
    assert np.abs(got[:, :rot // 2] - m * np.cos(a)).max() <= tol
    assert np.abs(got[:, rot // 2:] - m * np.sin(a)).max() <= tol


# ---------------------------------------------------------------- append

APPENDS = [
    # dt, new, ctx, hq, hkv, d, page, rot, inter, pad
    ("fp16", [1], [1], 4, 1, 128, 64, 128, False, 0),
    ("bf16", [1, 1, 1], [64, 65, 700], 8, 8, 128, 64, 128, False, 0),
    ("fp16", [5, 0, 64, 130, 1], [5, 0, 64, 200, 128], 6, 2, 128, 64, 64, True, 4),
    ("bf16", [3, 300, 0], [257, 556, 9], 3, 3, 64, 256, 16, False, 2),
    ("fp16", [2, 2, 2], [65, 129, 2], 14, 2, 64, 128, 64, True, 0),
    ("bf16", [67], [67], 2, 1, 128, 128, 0, False, 1)]


@pytest.mark.parametrize("dt,new,ctx,hq,hkv,d,page,rot,inter,pad", APPENDS)
@pytest.mark.parametrize("loud", [0.01, 30.0])
def test_append(P, dt, new, ctx, hq, hkv, d, page, rot, inter, pad, loud):
    """loud 0.01: older codes keep their scale; 30: it grows and they are requantized."""
    c = Case(11 + d + page, dt, new, ctx, hq, hkv, d, page, pad)
    qkv = c.act(hq + 2 * hkv, loud)
    table = None
    if rot:
        table = P.awq_rope_table(max(ctx) + 1, rot, base=500000.0)
    c.upload()
    x = qkv.to(DEV)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    out = torch.full((c.rows, hq, d), 7.0, dtype=DT[dt], device=DEV)
    got = append_fn(P, dt)(k, v, c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, cu_q=c.dcu, q=q, rope=table,
                           interleaved=inter, out=out)
    assert got is out
    th = table.cpu().numpy() if rot else None
    f = qkv.float().numpy()
    want = [a.copy() for a in (c.kc, c.vc, c.ks, c.vs)]
    R.append(*want, c.bt, c.ctx, c.cu, f[:, hq:hq + hkv], f[:, hq + hkv:], th, inter)
    same_cache(c, want)
    qr = f[:, :hq].copy()
    if rot:
        for b in range(len(ctx)):
            rr, first = R.positions(c.cu, c.ctx, b)
            p = first + np.arange(len(rr))
            qr[rr.start:rr.stop] = R.rotate(qr[rr.start:rr.stop], th[p], rot, inter)
    qr = torch.from_numpy(qr).to(DT[dt])
    qr[c.used:] = 7.0
    assert torch.equal(out.cpu().view(torch.int16), qr.view(torch.int16))
    # the same tokens again change nothing: the scales have grown already
    append_fn(P, dt)(k, v, c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, cu_q=c.dcu, rope=table, interleaved=inter)
    same_cache(c, want)


def test_append_in_place_and_single_rows(P):
    """q rotated onto itself; cu_q left out; one token a call over a page's end, against one call with all."""
    hq, hkv, d, page = 8, 2, 128, 64
    c = Case(5, "fp16", [1, 1], [63, 10], hq, hkv, d, page, fill=False, extra=4)
    c.bt = np.array([[0, 1], [2, 3]], np.int32)
    c.tokens(0, 0, 61)
    c.tokens(1, 0, 9)
    c.upload()
    table = P.awq_rope_table(80, d)
    th = table.cpu().numpy()
    want = [a.copy() for a in (c.kc, c.vc, c.ks, c.vs)]
    for i in range(4):
        c.ctx = np.array([62 + i, 10 + i], np.int32)
        x = c.act(hq + 2 * hkv, 1.0 + 3 * i)
        c.dctx.copy_(torch.from_numpy(c.ctx))
        dx = x.to(DEV)
        q = dx[:, :hq]
        out = P.awq_kv8_append(dx[:, hq:hq + hkv], dx[:, hq + hkv:], c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, q=q,
                               rope=table, out=q)
        assert out.data_ptr() == q.data_ptr()
        f = x.float().numpy()
        R.append(*want, c.bt, c.ctx, [0, 1, 2], f[:, hq:hq + hkv], f[:, hq + hkv:], th, False)
        same_cache(c, want)
        qr = torch.from_numpy(R.rotate(f[:, :hq], th[c.ctx - 1], d, False)).half()
        assert torch.equal(q.cpu().view(torch.int16), qr.view(torch.int16))


def test_append_odd_tokens(P):
    """inf and NaN, a position past the table, all-zero and tiny tokens, bf16's largest."""
    for dt in ("fp16", "bf16"):
        c = Case(21, dt, [70, 6], [90, 6], 2, 2, 64, 64)
        x = c.act(6)
        x[3, 2, 5] = float("inf")
        x[10, 4, 1] = float("nan")
        x[40, 3, :] = 0
        x[70:73, 2:] = 0
        if dt == "bf16":
            x[74, 2:] = 3.0e38
            x[60, 4, 0] = -3.3e38
        else:
            x[74, 2:] = 65504.0
            x[75, 3:] = 6e-8
        table = P.awq_rope_table(88, 32)
        c.upload()
        dx = x.to(DEV)
        q = append_fn(P, dt)(dx[:, 2:4], dx[:, 4:], c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, cu_q=c.dcu,
                             q=dx[:, :2], rope=table)
        f = x.float().numpy()
        want = [a.copy() for a in (c.kc, c.vc, c.ks, c.vs)]
        R.append(*want, c.bt, c.ctx, c.cu, f[:, 2:4], f[:, 4:], table.cpu().numpy(), False)
        same_cache(c, want)
        nan = torch.isnan(q).all(2).all(1).cpu().numpy()
        assert nan[68:70].all() and not nan[:68].any()          # positions 88 and 89 of a table of 88


@pytest.mark.parametrize("loud", [0.02, 40.0])
def test_append_keeps_scales_of_other_writers(P, loud):
    """Older tokens under scales that are no powers of two: kept (new codes by true quotients) or
    grown to a power of two."""
    for dt, page in (("bf16", 64), ("fp16", 128)):
        c = Case(25, dt, [3, 30, 1], [20, 90, 64], 4, 2, 128, page)
        c.ks *= c.rng.uniform(1.0, 1.999, c.ks.shape).astype(np.float32)
        c.vs *= c.rng.uniform(1.0, 1.999, c.vs.shape).astype(np.float32)
        x = c.act(8, loud)
        c.upload()
        dx = x.to(DEV)
        append_fn(P, dt)(dx[:, 4:6], dx[:, 6:], c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, cu_q=c.dcu)
        f = x.float().numpy()
        want = [a.copy() for a in (c.kc, c.vc, c.ks, c.vs)]
        R.append(*want, c.bt, c.ctx, c.cu, f[:, 4:6], f[:, 6:])
        same_cache(c, want)


def test_append_bad_pages_and_lengths(P):
    """Pages outside the cache and tokens past the table of pages are dropped, as are
    rows before position 0; nothing else changes."""
    c = Case(31, "fp16", [80, 40, 3, 9], [100, 20, 3, 3], 2, 2, 128, 64)
    c.bt[0, 0] = c.pages                     # first page of sequence 0: outside
    c.ctx[2] = 64 * c.bt.shape[1] + 2        # sequence 2: behind its row of the table
    x = c.act(4)
    c.upload()
    dx = x.to(DEV)
    P.awq_kv8_append(dx[:, :2], dx[:, 2:], c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, cu_q=c.dcu)
    f = x.float().numpy()
    want = [a.copy() for a in (c.kc, c.vc, c.ks, c.vs)]
    c.bt[2] = -1
    R.append(*want, c.bt, c.ctx, c.cu, f[:, :2], f[:, 2:])
    same_cache(c, want)


# ---------------------------------------------------------------- attention

def check_attn(c, q, out, lse, scale=None, kv=None, tokens_ok=None):
    scale = c.d ** -0.5 if scale is None else scale
    kc, vc, ks, vs = kv if kv is not None else (c.kc, c.vc, c.ks, c.vs)
    ref = R.attend(q.double().numpy(), kc, vc, ks, vs, c.bt, c.ctx, c.cu, scale)
    to, tl = R.bounds(*ref, c.d, torch.finfo(DT[c.dt]).eps)
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    u = c.used
    err = np.abs(got[:u] - ref[0][:u])
    assert np.isfinite(got[:u]).all()
    assert (err <= to[:u]).all(), (float((err / np.maximum(to[:u], 1e-300)).max()), np.argwhere(err > to[:u])[:4].tolist())
    empty = np.isneginf(ref[1][:u])
    assert np.array_equal(np.isneginf(glse[:u]), empty)
    el = np.abs(np.where(empty, 0, glse[:u]) - np.where(empty, 0, ref[1][:u]))
    assert (el <= tl[:u]).all(), float((el / tl[:u]).max())
    assert (got[u:] == 7.0).all() and (glse[u:] == 7.0).all()


def run_attn(P, c, q, max_q=None, scale=None, out=None, cu=True):
    out = torch.full((c.rows, c.hq, c.d), 7.0, dtype=DT[c.dt], device=DEV) if out is None else out
    lse = torch.full((c.rows, c.hq), 7.0, device=DEV)
    got = attn_fn(P, c.dt)(q, c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, cu_q=c.dcu if cu else None, max_q=max_q,
                           scale=scale, out=out, lse=lse)
    assert got is out
    return out, lse


ATTNS = [
    # dt, new, ctx, hq, hkv, d, page, pad
    ("fp16", [1], [1], 1, 1, 128, 64, 0),
    ("bf16", [1, 1, 1, 1], [1, 64, 65, 1000], 8, 2, 128, 64, 0),
    ("fp16", [1, 1, 1], [127, 2, 513], 32, 1, 64, 128, 2),           # 32 heads of one: two tiles
    ("bf16", [1, 0, 1], [300, 40, 0], 14, 2, 128, 256, 3),           # idle; empty context
    ("fp16", [5, 3, 0, 9], [5, 260, 0, 4], 24, 8, 64, 64, 1),        # ctx < n: rows that see nothing
    ("bf16", [33, 130], [33, 450], 4, 4, 128, 64, 0),
    ("fp16", [200, 1, 17], [200, 700, 1100], 8, 2, 128, 64, 5),
    ("bf16", [64, 65], [64, 321], 6, 2, 64, 256, 0),
    ("fp16", [70], [2000], 7, 1, 128, 128, 0)]


@pytest.mark.parametrize("dt,new,ctx,hq,hkv,d,page,pad", ATTNS)
@pytest.mark.parametrize("known", [True, False])
def test_attention(P, dt, new, ctx, hq, hkv, d, page, pad, known):
    c = Case(40 + d + page + len(new), dt, new, ctx, hq, hkv, d, page, pad)
    c.upload()
    q = c.act(hq, 1.3)
    big = torch.zeros(c.rows, hq + 3, d, dtype=DT[dt])
    big[:, 1:1 + hq] = q
    out, lse = run_attn(P, c, big.to(DEV)[:, 1:1 + hq], max_q=max(new) if known else 1 << 20)
    check_attn(c, q, out, lse)
    again = run_attn(P, c, q.to(DEV), max_q=max(new) if known else 1 << 20)
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse, again[1])
    # a wrong idea of the most rows changes the kernel, not the result
    out, lse = run_attn(P, c, q.to(DEV), max_q=1)
    check_attn(c, q, out, lse)


@pytest.mark.parametrize("b", [65, 130])
def test_attention_many_sequences_many_columns(P, b):
    """More than 64 sequences in tiles of 128 columns, one of them long enough to be split."""
    rng = np.random.default_rng(b)
    new = rng.integers(0, 20, b)
    new[3], new[b - 1] = 40, 33
    ctx = new + rng.integers(0, 90, b)
    ctx[b - 1] += 2500
    c = Case(b + 7, "fp16", new, ctx, 4, 1, 64, 64)
    c.upload()
    q = c.act(4)
    out, lse = run_attn(P, c, q.to(DEV), max_q=40)
    check_attn(c, q, out, lse)


@pytest.mark.parametrize("b", [63, 64, 65, 200])
def test_attention_many_sequences(P, b):
    rng = np.random.default_rng(b)
    ctx = rng.integers(0, 200, b)
    ctx[b // 2] = 3000
    c = Case(b, "fp16", [1] * b, ctx, 4, 2, 64, 64)
    c.upload()
    q = c.act(4)
    out, lse = run_attn(P, c, q.to(DEV), cu=False)
    check_attn(c, q, out, lse)
    new = rng.integers(0, 4, b)
    c = Case(b + 1, "bf16", new, ctx + new, 4, 1, 128, 64)
    c.upload()
    q = c.act(4)
    out, lse = run_attn(P, c, q.to(DEV), max_q=3)
    check_attn(c, q, out, lse)


def test_attention_so_many_sequences_that_two_waves_take_a_tile(P):
    rng = np.random.default_rng(300)
    ctx = rng.integers(0, 40, 300)
    ctx[17], ctx[299] = 2000, 700
    for hq, once in ((8, True), (16, False)):
        new = np.ones(300, np.int64) if once else rng.integers(0, 3, 300)
        c = Case(301 + hq, "bf16" if once else "fp16", new, np.maximum(ctx, new), hq, 8, 64, 64)
        c.upload()
        q = c.act(hq)
        out, lse = run_attn(P, c, q.to(DEV), max_q=int(new.max()), cu=not once)
        check_attn(c, q, out, lse)


def test_attention_joins_hundreds_of_parts(P):
    """One context so much longer than thousands of others that its column comes in some 300 parts."""
    ctx = np.ones(2050, np.int64)
    ctx[2000] = 80000
    c = Case(2050, "bf16", [1] * 2050, ctx, 1, 1, 64, 64)
    c.upload()
    q = c.act(1)
    out, lse = run_attn(P, c, q.to(DEV), cu=False)
    check_attn(c, q, out, lse)


@pytest.mark.parametrize("new", [1, 6, 40])
def test_attention_long_context_is_split(P, new):
    c = Case(77, "fp16", [new, new], [9000, 700], 4, 1, 128, 64)
    c.upload()
    q = c.act(4)
    assert P.awq_attn_kv8_workspace_size(2, c.rows, 4, 1, 128, 64, c.bt.shape[1], new) > 0
    out, lse = run_attn(P, c, q.to(DEV), max_q=new)
    check_attn(c, q, out, lse)


@pytest.mark.parametrize("d,page", [(64, 64), (128, 256)])
def test_attention_split_in_wide_tiles(P, d, page):
    """Enough rows and heads for tiles of 128 columns, contexts long enough to be split between them."""
    c = Case(78, "bf16", [200, 150, 3], [3000, 2300, 70], 32, 32, d, page, pad=1)
    c.upload()
    q = c.act(32)
    out, lse = run_attn(P, c, q.to(DEV), max_q=200)
    check_attn(c, q, out, lse)
    again = run_attn(P, c, q.to(DEV), max_q=200)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("b", [64, 100])
def test_attention_many_sequences_in_wide_tiles(P, b):
    rng = np.random.default_rng(b)
    new = rng.integers(0, 20, b)
    new[3], new[b - 1] = 40, 33
    ctx = new + rng.integers(0, 90, b)
    ctx[b - 1] += 2500
    c = Case(b + 9, "bf16", new, ctx, 8, 2, 64, 64)
    c.upload()
    q = c.act(8)
    out, lse = run_attn(P, c, q.to(DEV), max_q=40)
    check_attn(c, q, out, lse)


def test_attention_bad_page_and_odd_query_in_wide_tiles(P):
    """The same isolation in tiles of 128 columns: a page outside the cache is seen by later rows only."""
    c = Case(79, "fp16", [140, 60], [2400, 2200], 16, 16, 128, 64)
    q = c.act(16)
    c.upload()
    want = run_attn(P, c, q.to(DEV), max_q=140)
    bt = c.bt.copy()
    bt[0, 36] = -7                                      # positions 2304 ..: rows 44 on of sequence 0
    c.dbt.copy_(torch.from_numpy(bt))
    bad = q.clone()
    bad[150, 3, 2] = float("nan")
    out, lse = run_attn(P, c, bad.to(DEV), max_q=140)
    odd = torch.zeros(c.rows, 16, dtype=torch.bool, device=DEV)
    odd[44:140] = True
    odd[150, 3] = True
    assert torch.isnan(out[odd]).all() and torch.isnan(lse[odd]).all()
    assert torch.equal(out[~odd], want[0][~odd]) and torch.equal(lse[~odd], want[1][~odd])


def test_attention_scales_far_apart(P):
    """Value scales from 2^-40 to 2^40 in one context, key scales likewise, peaked scores."""
    c = Case(91, "bf16", [1, 4], [640, 300], 8, 2, 128, 64)
    rng = np.random.default_rng(1)
    c.vs[:] = 2.0 ** rng.choice([-40, -20, -3, 10, 40], c.vs.shape)
    c.ks[:] = 2.0 ** rng.choice([-64, -9, -5], c.ks.shape)
    c.upload()
    q = c.act(8, 2.0)
    out, lse = run_attn(P, c, q.to(DEV), max_q=4)
    check_attn(c, q, out, lse)


def test_attention_bad_pages_give_nan(P):
    """A page outside the cache, or a context longer than the table of pages: NaN for the
    rows that see it, the others as they are."""
    c = Case(93, "fp16", [1, 1, 70, 1], [100, 200, 130, 5], 4, 2, 64, 64)
    q = c.act(4)
    c.upload()
    want = run_attn(P, c, q.to(DEV), max_q=70)
    bt, ctx = c.bt.copy(), c.ctx.copy()
    bt[0, 1] = -1
    bt[2, 1] = c.pages                                  # positions 64 ..: rows 4 on of sequence 2 see it
    c.dbt.copy_(torch.from_numpy(bt))
    ctx[3] = 64 * bt.shape[1] + 1
    c.dctx.copy_(torch.from_numpy(ctx))
    out, lse = run_attn(P, c, q.to(DEV), max_q=70)
    nan = torch.isnan(out).all(2).cpu().numpy()
    seen = np.zeros(c.rows, bool)
    seen[0] = seen[-1] = True
    seen[2 + 4:2 + 70] = True                           # row 2 + i stands at 60 + i
    assert np.array_equal(nan, np.repeat(seen[:, None], 4, 1))
    keep = torch.from_numpy(~seen).to(DEV)
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


def test_poisoned_token_is_seen_by_later_rows_only(P):
    hq, hkv, d = 4, 2, 64
    c = Case(95, "fp16", [80], [80], hq, hkv, d, 64, fill=False)
    x = c.act(hq + 2 * hkv)
    y = x.clone()
    y[70, hq + hkv, 3] = float("nan")                   # v of head 0
    outs = []
    for z in (x, y):
        c.upload()
        dz = z.to(DEV)
        P.awq_kv8_append(dz[:, hq:hq + hkv], dz[:, hq + hkv:], c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, cu_q=c.dcu)
        outs.append(run_attn(P, c, dz[:, :hq], max_q=80)[0].float().cpu().numpy())
    nan = np.isnan(outs[1]).all(2)
    assert nan[70:, :2].all() and not nan[:70].any() and not nan[:, 2:].any()
    # the scale of its page is another, as the token does not count for it: compare the page before it
    assert np.array_equal(outs[0][:64], outs[1][:64])


@pytest.mark.parametrize("new", [3, 5, 50])
def test_odd_queries_stay_alone(P, new):
    """NaN and inf in one row's query change that row and head only."""
    c = Case(98, "bf16", [new, 2], [400, 66], 4, 1, 128, 64)
    c.upload()
    q = c.act(4)
    want = run_attn(P, c, q.to(DEV), max_q=new)
    bad = q.clone()
    bad[1, 2, 7] = float("nan")
    bad[new, 0, 0] = float("inf")
    out, lse = run_attn(P, c, bad.to(DEV), max_q=new)
    odd = torch.zeros(c.rows, 4, dtype=torch.bool, device=DEV)
    odd[1, 2] = odd[new, 0] = True
    assert torch.isnan(out[odd]).all() and torch.isnan(lse[odd]).all()
    assert torch.equal(out[~odd], want[0][~odd]) and torch.equal(lse[~odd], want[1][~odd])


def test_no_rows_and_no_sequences(P):
    """Empty calls write nothing: no rows, no sequences, an empty block table."""
    c = Case(100, "fp16", [0, 0], [70, 3], 4, 2, 64, 64)
    c.upload()
    none = torch.empty(0, 4, 64, dtype=torch.float16, device=DEV)
    kv = torch.empty(0, 2, 64, dtype=torch.float16, device=DEV)
    assert P.awq_kv8_append(kv, kv, c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, cu_q=c.dcu, q=none).shape == (0, 4, 64)
    assert P.awq_attn_kv8(none, c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, cu_q=c.dcu).shape == (0, 4, 64)
    same_cache(c, (c.kc, c.vc, c.ks, c.vs))
    # rows, but every sequence idle: the rows are nobody's
    q = torch.randn(5, 4, 64, device=DEV).half()
    out, lse = torch.full_like(q, 7.0), torch.full((5, 4), 7.0, device=DEV)
    P.awq_attn_kv8(q, c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, cu_q=c.dcu, out=out, lse=lse)
    P.awq_kv8_append(q[:, :2], q[:, 2:], c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, cu_q=c.dcu)
    assert (out == 7).all() and (lse == 7).all()
    same_cache(c, (c.kc, c.vc, c.ks, c.vs))
    # no pages at all: every row sees nothing (ctx 0) or NaN (ctx 1)
    ctx = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    bt = torch.empty(2, 0, dtype=torch.int32, device=DEV)
    out, lse = torch.full_like(q[:2], 7.0), torch.full((2, 4), 7.0, device=DEV)
    P.awq_attn_kv8(q[:2], c.dk, c.dv, c.dks, c.dvs, bt, ctx, out=out, lse=lse)
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()


@pytest.mark.parametrize("extra", [1, 40])
def test_rows_within_the_block_table_are_kept(P, extra):
    """A sequence longer than its row of the block table: NaN for the rows that stand behind it only."""
    c = Case(102, "fp16", [30 + extra, 3], [640 + extra, 100], 4, 1, 128, 64)
    assert c.bt.shape[1] == 11
    q = c.act(4)
    c.upload()
    want = run_attn(P, c, q.to(DEV), max_q=30 + extra)
    c.dbt = c.dbt[:, :10].contiguous()
    for max_q in (30 + extra, 1):
        out, lse = run_attn(P, c, q.to(DEV), max_q=max_q)
        lost = torch.zeros(c.rows, dtype=torch.bool, device=DEV)
        lost[30:30 + extra] = True
        assert torch.isnan(out[lost]).all() and torch.isnan(lse[lost]).all()
        assert torch.isfinite(out[~lost]).all()
        assert (out[~lost].double() - want[0][~lost].double()).abs().max() <= 2.0 ** -9 * want[0].double().abs().max()


def test_attention_peaked_and_scaled(P):
    """Scores of hundreds (the running maximum moves at almost every step) and another softmax scale."""
    c = Case(97, "fp16", [3, 90], [900, 500], 4, 2, 128, 64)
    c.upload()
    q = c.act(4, 25.0)
    out, lse = run_attn(P, c, q.to(DEV), max_q=90, scale=0.2)
    check_attn(c, q, out, lse, scale=0.2)


@pytest.mark.parametrize("new", [1, 3, 40])
@pytest.mark.parametrize("gap", [12.0, 24.3])
def test_attention_first_token_outweighs_all(P, new, gap):
    """One token whose score exceeds every other by a factor of 2^gap, its v zero: the result is the
    others' small share, which must keep its relative precision."""
    c = Case(96, "fp16", [new], [3000], 4, 1, 128, 64)
    c.kc[:] = 0
    c.kc[c.bt[0, 0], 0, 0] = R.encode(np.full(128, 1.0))
    c.ks[:] = 1.0
    c.vc[:] = R.encode(np.full(c.vc.shape, 3.0))
    c.vc[c.bt[0, 0], 0, :, 0] = 0
    c.vs[:] = 1.0
    c.upload()
    q = torch.full((new, 4, 128), gap * np.log(2) / 128 ** 0.5).half()
    out, lse = run_attn(P, c, q.to(DEV), max_q=new)
    ref = R.attend(q.double().numpy(), c.kc, c.vc, c.ks, c.vs, c.bt, c.ctx, c.cu, 128 ** -0.5)
    # scores of a few tens, so weights within 2^-14; fp16 outputs within half a step, or of a subnormal one
    tol = 2.0 ** -13 * np.abs(ref[0]) + np.maximum(2.0 ** -11 * np.abs(ref[0]), 2.0 ** -25)
    assert (np.abs(out.double().cpu().numpy() - ref[0]) <= tol).all()
    check_attn(c, q, out, lse)


def test_cache_beyond_32_bit_offsets(P):
    """Pages that start behind 4 GiB of the cache."""
    hq, hkv, d, page = 8, 8, 128, 64
    pages = 66000                                       # 65536 bytes a page: 4.3 GB for k, as much for v
    kc, vc, ks, vs = P.kv8_cache(pages, hkv, d, page, device=DEV)
    c = Case(99, "fp16", [150, 1], [150, 1], hq, hkv, d, page, fill=False)
    high = np.arange(pages - c.pages, pages)
    x = c.act(hq + 2 * hkv).to(DEV)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    c.upload()
    P.awq_kv8_append(k, v, c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, cu_q=c.dcu)
    want = run_attn(P, c, q, max_q=150)
    live = c.bt.copy()
    live[(live >= 0) & (live < c.pages)] += pages - c.pages
    bt = dev(live)
    P.awq_kv8_append(k, v, kc, vc, ks, vs, bt, c.dctx, cu_q=c.dcu)
    out = torch.full_like(want[0], 7.0)
    P.awq_attn_kv8(q, kc, vc, ks, vs, bt, c.dctx, cu_q=c.dcu, max_q=150, out=out)
    assert torch.equal(out, want[0])
    used = [int(p) for p in c.bt[0, :3]] + [int(c.bt[1, 0])]
    for p in used:
        assert torch.equal(ks[high[p]], c.dks[p])


def test_workspace_and_outputs_stay_inside(P):
    c = Case(101, "fp16", [1, 4, 130], [5000, 800, 300], 8, 2, 128, 64, pad=2)
    c.upload()
    q = c.act(8)
    need = P.awq_attn_kv8_workspace_size(3, c.rows, 8, 2, 128, 64, c.bt.shape[1], 130)
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    out = torch.full((c.rows + 2, 8, 128), 7.0, dtype=torch.float16, device=DEV)
    lse = torch.full((c.rows + 2, 8), 7.0, device=DEV)
    P.awq_attn_kv8(q.to(DEV), c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, cu_q=c.dcu, max_q=130, out=out[1:-1],
                   lse=lse[1:-1], workspace=ws[256:256 + need])
    check_attn(c, q, out[1:-1], lse[1:-1])
    assert (ws[:256] == 0xA5).all() and (ws[256 + need:] == 0xA5).all()
    assert (out[0] == 7).all() and (out[-1] == 7).all() and (lse[0] == 7).all() and (lse[-1] == 7).all()


def test_two_streams(P):
    cases = [Case(103 + i, "fp16", [1, 2], [6000, 900], 8, 2, 128, 64) for i in range(2)]
    qs, want = [], []
    for c in cases:
        c.upload()
        qs.append(c.act(8).to(DEV))
        want.append(run_attn(P, c, qs[-1], max_q=2))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for c, q, s in zip(cases, qs, streams):
        with torch.cuda.stream(s):
            got.append([run_attn(P, c, q, max_q=2) for _ in range(5)])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for o, l in g:
            assert torch.equal(o, w[0]) and torch.equal(l, w[1])


def test_captured_step_follows_the_lengths(P):
    """Append and attention captured once and replayed while the sequences grow: the plan is
    made on the device, so a replay uses the lengths it finds."""
    hq, hkv, d, page = 8, 2, 128, 64
    c = Case(107, "bf16", [1, 1, 1], [60, 1000, 5], hq, hkv, d, page, extra=9)
    wide = np.zeros((3, 20), np.int32)
    free = [p for p in range(c.pages) if p not in set(c.bt[0, :1]) | set(c.bt[1, :16]) | set(c.bt[2, :1])]
    for b, n in enumerate((1, 16, 1)):
        wide[b, :n] = c.bt[b, :n]
        wide[b, n] = free.pop()
    c.bt = wide
    c.upload()
    table = P.awq_rope_table(1200, d)
    x = c.act(hq + 2 * hkv).to(DEV)
    q_out = torch.zeros(3, hq, d, dtype=torch.bfloat16, device=DEV)
    out, lse = torch.zeros_like(q_out), torch.zeros(3, hq, device=DEV)
    ws = torch.empty(P.awq_attn_kv8_workspace_size(3, 3, hq, hkv, d, page, 20, 1), dtype=torch.uint8, device=DEV)

    def step():
        P.awq_kv8_append_bf16(x[:, hq:hq + hkv], x[:, hq + hkv:], c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx,
                              q=x[:, :hq], rope=table, out=q_out)
        P.awq_attn_kv8_bf16(q_out, c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, out=out, lse=lse, workspace=ws)

    start = [t.clone() for t in (c.dk.view(torch.uint8), c.dv.view(torch.uint8), c.dks, c.dvs, c.dctx, x)]

    def reset():
        for t, s in zip((c.dk.view(torch.uint8), c.dv.view(torch.uint8), c.dks, c.dvs, c.dctx, x), start):
            t.copy_(s)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    runs = []
    for replay in (False, True):
        reset()
        seen = []
        for i in range(10):
            c.dctx.add_(1)
            x.mul_(1.0 + 0.25 * (i % 3))
            graph.replay() if replay else step()
            seen.append((out.clone(), lse.clone(), c.dks.clone()))
        torch.cuda.synchronize()
        runs.append(seen + [(c.dk.view(torch.uint8).clone(), c.dv.view(torch.uint8).clone(), c.dvs.clone())])
    for a, b in zip(*runs):
        for s, t in zip(a, b):
            assert torch.equal(s, t)


def test_decoder_attention_block(P):
    """The entries as a layer uses them: q, k and v from one group call of 4-bit linears, append
    with rotation, attention, the o linear; a prompt and then single tokens.  Every stage is
    checked against the definition on the stage's own inputs."""
    hidden, hq, hkv, d, g = 512, 4, 2, 128, 128
    widths = (hq * d, hkv * d, hkv * d)
    packs = []
    for i, n in enumerate((*widths, hidden)):
        k = hidden if i < 3 else hq * d
        qw, sc, qz, _ = O.pack_int4(S.weights(n, k, 0.04, 700 + i), None, g)
        packs.append((qw, sc, qz))
    devp = [tuple(dev(a.view(np.int32)) if a.dtype == np.uint32 else dev(a) for a in p) for p in packs]
    table = P.awq_rope_table(300, d, base=500000.0)
    th = table.cpu().numpy()
    cache = P.kv8_cache(12, hkv, d, 64, device=DEV)
    host = [np.zeros((12, hkv, 64, d), np.uint8), np.zeros((12, hkv, d, 64), np.uint8),
            np.ones((12, hkv), np.float32), np.ones((12, hkv), np.float32)]
    for t, a in zip(cache, host):
        (t.view(torch.uint8) if a.dtype == np.uint8 else t).copy_(torch.from_numpy(a))
    bt = np.array([[5, 0, 7], [2, 11, 3]], np.int32)
    dbt = dev(bt)
    ctx = np.zeros(2, np.int32)
    for step, new in enumerate(((130, 41), (1, 1), (1, 1), (4, 0))):
        rows = sum(new)
        ctx = ctx + np.array(new, np.int32)
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        x = S.activations(rows, hidden, 800 + step, S.outlier_channels(hidden, 0.01, 3), 10.0)
        xd = dev(x)
        q, k, v = P.awq_linear_w4a16_group([(xd, *p, None, None) for p in devp[:3]], g=g)
        q, k, v = q.view(rows, hq, d), k.view(rows, hkv, d), v.view(rows, hkv, d)
        dcu, dctx = dev(cu), dev(ctx)
        qr = P.awq_kv8_append(k, v, *cache, dbt, dctx, cu_q=dcu, q=q, rope=table)
        lse = torch.empty(rows, hq, device=DEV)
        o = P.awq_attn_kv8(qr, *cache, dbt, dctx, cu_q=dcu, max_q=max(new), lse=lse)
        y = P.awq_linear_w4a16(o.view(rows, hq * d), *devp[3], g=g)
        R.append(*host, bt, ctx, cu, k.float().cpu().numpy(), v.float().cpu().numpy(), th, False)
        for t, a in zip(cache, host):
            got = (t.view(torch.uint8) if a.dtype == np.uint8 else t).cpu().numpy()
            assert np.array_equal(got, a), step
        c = Case.__new__(Case)
        c.dt, c.d, c.used, c.bt, c.ctx, c.cu = "fp16", d, rows, bt, ctx, cu
        check_attn(c, qr.cpu(), o, lse, kv=host)
        ok, worst, _ = O.check_linear(y.cpu().numpy(), O.linear_ref(o.view(rows, hq * d).cpu().numpy(), *packs[3], None,
                                                                    hq * d, g))
        assert ok, (step, worst)
