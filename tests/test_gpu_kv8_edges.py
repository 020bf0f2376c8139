"""Edges of the 8-bit paged KV cache on the GPU: what a page outside the cache stands on, the
numerics of far-apart scales and weights in the widest tiles, callers in several threads, far
rotary positions."""
from __future__ import annotations

import numpy as np
import pytest

from tests import kv8_ref as R
from tests.test_gpu_kv8 import DEV, P, Case, attn_fn, check_attn, run_attn  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


# ---------------------------------------------------------------- pages outside the cache

def leave_page_0(c):
    """Moves what a sequence holds in page 0 of the cache to a page that none holds."""
    used = {int(p) for i, n in enumerate(c.ctx) for p in c.bt[i, :max(1, -(-int(n) // c.page))]}
    if 0 not in used:
        return
    free = max(p for p in range(c.pages) if p not in used)
    at = np.argwhere(c.bt == 0)
    for i, j in at:
        if j < max(1, -(-int(c.ctx[i]) // c.page)):
            c.bt[i, j] = free
    for a in (c.kc, c.vc, c.ks, c.vs):
        a[[0, free]] = a[[free, 0]]


FORMS = [
    # dt, new, ctx, hq, hkv, d, the entry of sequence 0 that names no page, its first row that sees it
    ("fp16", [6, 2], [130, 70], 4, 2, 128, 2, 4),                 # one tile of 16 columns
    ("bf16", [6, 2], [8964, 70], 4, 2, 128, 140, 2),              # the same in parts
    ("bf16", [6, 0], [130, 9], 16, 2, 64, 2, 4),                  # tiles of 16 columns of one sequence
    ("fp16", [40, 3], [2970, 100], 4, 1, 64, 46, 14),             # tiles of 32 columns
    ("fp16", [70, 1], [130, 200], 4, 2, 128, 1, 4),               # tiles of 128 columns
    ("bf16", [140, 60], [2400, 2200], 64, 64, 64, 36, 44)]        # the same in parts


@pytest.mark.parametrize("dt,new,ctx,hq,hkv,d,entry,sees", FORMS)
@pytest.mark.parametrize("scale0", [0.0, float("nan"), float("inf"), 1e-40])
def test_bad_page_whatever_page_0_holds(P, dt, new, ctx, hq, hkv, d, entry, sees, scale0):  # noqa: F811
    """Page 0 belongs to nobody and its scales were never set: rows that do not see the page outside the
    cache keep their results, those that see it are NaN."""
    c = Case(200 + d + len(ctx), dt, new, ctx, hq, hkv, d, 64)
    leave_page_0(c)
    c.ks[0] = c.vs[0] = scale0
    c.upload()
    q = c.act(hq).to(DEV)
    want = run_attn(P, c, q, max_q=max(new))
    assert torch.isfinite(want[0]).all() and torch.isfinite(want[1]).all()
    for outside in (-1, c.pages):
        bt = c.bt.copy()
        bt[0, entry] = outside
        c.dbt.copy_(torch.from_numpy(bt))
        out, lse = run_attn(P, c, q, max_q=max(new))
        odd = torch.zeros(c.rows, dtype=torch.bool, device=DEV)
        odd[sees:new[0]] = True
        assert torch.isnan(out[odd]).all() and torch.isnan(lse[odd]).all()
        assert torch.equal(out[~odd], want[0][~odd]) and torch.equal(lse[~odd], want[1][~odd])


# ---------------------------------------------------------------- scales at the ends of their range

@pytest.mark.parametrize("new,ctx,hq,hkv", [([3], [200], 4, 2), ([3], [9000], 4, 2), ([40], [2500], 4, 1),
                                            ([70], [200], 4, 2), ([130], [2500], 72, 72)])
@pytest.mark.parametrize("exponent", [-64, 120])
def test_value_scales_at_their_ends(P, new, ctx, hq, hkv, exponent):  # noqa: F811
    """Every value scale 2^-64 (a page of zeros as the append writes it) or 2^120 (of bf16's largest values), in each
    tile form, whole and in parts."""
    c = Case(240, "bf16", new, ctx, hq, hkv, 64, 64)
    c.vs[:] = 2.0 ** exponent
    small = np.abs(R.CODE[c.vc]) < 8                    # values within bf16: 448 * 2^120 is not
    c.vc = np.where(small, c.vc, R.encode(np.full(c.vc.shape, 2.0))).astype(np.uint8)
    c.upload()
    q = c.act(hq, 1.3)
    out, lse = run_attn(P, c, q.to(DEV), max_q=new[0])
    ref = R.attend(q.double().numpy(), c.kc, c.vc, c.ks, c.vs, c.bt, c.ctx, c.cu, 64 ** -0.5)
    # attend()'s bounds take the argument of exp2 for one of at most 2 smag + 128; with a scale of 2^120 it is at
    # most 2 smag + 240, and the rounding 2^-23 * 112 more, which counts twice in a weight
    more = 2.0 ** -23 * 112
    to, tl = R.bounds(*ref, 64, torch.finfo(torch.bfloat16).eps)
    to, tl = to + 2 * more * 1.01 * ref[2], tl + more
    assert (np.abs(out.double().cpu().numpy() - ref[0]) <= to).all()
    assert (np.abs(lse.double().cpu().numpy() - ref[1]) <= tl).all()


# ---------------------------------------------------------------- rotary tables

@pytest.mark.parametrize("factor", [0.25, 1.0, 1.5])
def test_yarn_magnitude_starts_at_one(P, factor):  # noqa: F811
    """The magnitude 0.1 ln(factor) + 1 is for contexts that grow; up to factor 1 it is 1."""
    table = P.awq_rope_table(100, 64, scaling="yarn", factor=factor, low=1.0, high=32.0, trained=4096)
    m = 0.1 * np.log(factor) + 1 if factor > 1 else 1.0
    # position 0: cos 0 = 1 and sin 0 = 0 exactly, so m rounded to fp32 (half a step is 2^-24 of it)
    assert (table[0, 32:] == 0).all() and (table[0, :32].double() - m).abs().max().item() <= 2.0 ** -24 * m
    # cos^2 + sin^2 = m^2: each within 2^-22 m, so their squares' sum within 2 * 2^-22 * 1.5 m^2
    t = table.double().cpu()
    assert ((t[:, :32] ** 2 + t[:, 32:] ** 2) - m * m).abs().max().item() <= 3 * 2.0 ** -22 * m * m


@pytest.mark.parametrize("positions,rot,base", [(1 << 24, 16, 10000.0), (1 << 27, 16, 500000.0), ((1 << 31) - 1, 2, 10000.0)])
def test_rope_table_far_positions(P, positions, rot, base):  # noqa: F811
    """The last rows of long tables, against 80-bit floats: 2 ulp of 1 (2^-22) and the angle's own 2^-49 p f beyond
    p f = 2^24."""
    table = P.awq_rope_table(positions, rot, base=base)
    n = 20000
    got = table[-n:].cpu().numpy().astype(np.float64)
    del table
    p = np.arange(positions - n, positions).astype(np.longdouble)
    f = np.longdouble(base) ** (np.arange(rot // 2).astype(np.longdouble) * -2 / rot)
    a = p[:, None] * f
    tol = 2.0 ** -22 + np.where(a > 2.0 ** 24, 2.0 ** -49 * a.astype(np.float64), 0)
    assert (np.abs(got[:, :rot // 2] - np.cos(a)) <= tol).all()
    assert (np.abs(got[:, rot // 2:] - np.sin(a)) <= tol).all()


# ---------------------------------------------------------------- numerics of the 128-column tiles

WIDE = [
    # new, ctx, hq, hkv, d: over 64 columns on contexts of at most 32 steps; then at least 144 tiles
    # over all heads on longer ones, in parts
    ([40, 1], [300, 640], 8, 2, 128),
    ([130, 3], [3000, 70], 72, 72, 64)]


@pytest.mark.parametrize("new,ctx,hq,hkv,d", WIDE)
def test_wide_tiles_scales_far_apart(P, new, ctx, hq, hkv, d):  # noqa: F811
    """Value scales from 2^-40 to 2^40 in one context, key scales likewise, peaked scores."""
    c = Case(211 + d, "bf16", new, ctx, hq, hkv, d, 64)
    rng = np.random.default_rng(2)
    c.vs[:] = 2.0 ** rng.choice([-40, -20, -3, 10, 40], c.vs.shape)
    c.ks[:] = 2.0 ** rng.choice([-64, -9, -5], c.ks.shape)
    c.upload()
    q = c.act(hq, 2.0)
    out, lse = run_attn(P, c, q.to(DEV), max_q=max(new))
    check_attn(c, q, out, lse)


@pytest.mark.parametrize("new,ctx,hq,hkv,d", [([40], [2000], 4, 1, 128), ([130], [3000], 72, 72, 64)])
@pytest.mark.parametrize("gap", [12.0, 24.3])
def test_wide_tiles_first_token_outweighs_all(P, new, ctx, hq, hkv, d, gap):  # noqa: F811
    """One token whose score exceeds every other by a factor of 2^gap, its v zero and the others' v all
    alike: the bound is relative to the small share that is left of them."""
    c = Case(215, "fp16", new, ctx, hq, hkv, d, 64)
    c.kc[:] = 0
    c.kc[c.bt[0, 0], :, 0] = R.encode(np.full(d, 1.0))
    c.ks[:] = 1.0
    c.vc[:] = R.encode(np.full(c.vc.shape, 3.0))
    c.vc[c.bt[0, 0], :, :, 0] = 0
    c.vs[:] = 1.0
    c.upload()
    q = torch.full((new[0], hq, d), gap * np.log(2) / d ** 0.5).half()
    out, lse = run_attn(P, c, q.to(DEV), max_q=new[0])
    check_attn(c, q, out, lse)


# ---------------------------------------------------------------- callers, padded batches, graphs

def test_two_threads(P):  # noqa: F811
    """Append and attention from two threads at once, a stream each, with the binding's own workspaces."""
    import threading
    cases, xs, want = [], [], []
    for i in range(2):
        c = Case(230 + i, "fp16", [2, 1], [6000, 900], 8, 2, 128, 64)
        c.upload()
        cases.append(c)
        xs.append(c.act(12).to(DEV))

    def step(c, x):
        P.awq_kv8_append(x[:, 8:10], x[:, 10:], c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, cu_q=c.dcu)
        return run_attn(P, c, x[:, :8], max_q=2)

    for c, x in zip(cases, xs):
        want.append(step(c, x))                       # the same tokens again change nothing
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    got[i].append(step(cases[i], xs[i]))
            s.synchronize()
        except BaseException as e:                    # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for g, w in zip(got, want):
        assert len(g) == 20
        for o, l in g:
            assert torch.equal(o, w[0]) and torch.equal(l, w[1])


@pytest.mark.parametrize("ctx", [[70, 3, 400], [70, 3, 9000]])
def test_padded_batch_of_single_tokens(P, ctx):  # noqa: F811
    """Without cu_q, more rows than sequences: those behind the last one are neither read nor written."""
    hq, hkv, d = 8, 2, 128
    c = Case(250, "fp16", [1, 1, 1], ctx, hq, hkv, d, 64, pad=3)
    x = c.act(hq + 2 * hkv)
    x[3:] = float("nan")
    c.upload()
    dx = x.to(DEV)
    q_out = torch.full((6, hq, d), 7.0, dtype=torch.float16, device=DEV)
    P.awq_kv8_append(dx[:, hq:hq + hkv], dx[:, hq + hkv:], c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, q=dx[:, :hq],
                     out=q_out)
    f = x.float().numpy()
    R.append(c.kc, c.vc, c.ks, c.vs, c.bt, c.ctx, c.cu, f[:, hq:hq + hkv], f[:, hq + hkv:])
    for got, want in zip(c.cache(), (c.kc, c.vc, c.ks, c.vs)):
        assert np.array_equal(got, want)
    assert torch.equal(q_out[:3], dx[:3, :hq]) and (q_out[3:] == 7).all()
    out, lse = run_attn(P, c, q_out, cu=False)
    check_attn(c, q_out.cpu(), out, lse)


def test_captured_prompts_follow_the_lengths(P):  # noqa: F811
    """Append and attention over 128-column tiles and their joins, captured once and replayed with other rows per
    sequence and other contexts, eager calls with the same workspace between the replays."""
    hq, hkv, d = 32, 32, 64
    steps = [([200, 150, 3], [2900, 2300, 70]), ([3, 310, 40], [3, 3000, 2800]), ([0, 0, 353], [9, 0, 3000]),
             ([353, 0, 0], [353, 64, 0])]
    base = Case(260, "bf16", [200, 150, 3], [3000, 3000, 3000], hq, hkv, d, 64)
    base.upload()
    table = P.awq_rope_table(3000, d)
    x = base.act(hq + 2 * hkv).to(DEV)
    rows = x.shape[0]
    need = P.awq_attn_kv8_workspace_size(3, rows, hq, hkv, d, 64, base.bt.shape[1], rows)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    q_out = torch.zeros(rows, hq, d, dtype=torch.bfloat16, device=DEV)
    out, lse = torch.zeros_like(q_out), torch.zeros(rows, hq, device=DEV)

    def step():
        P.awq_kv8_append_bf16(x[:, hq:hq + hkv], x[:, hq + hkv:], base.dk, base.dv, base.dks, base.dvs, base.dbt,
                              base.dctx, cu_q=base.dcu, q=x[:, :hq], rope=table, out=q_out)
        P.awq_attn_kv8_bf16(q_out, base.dk, base.dv, base.dks, base.dvs, base.dbt, base.dctx, cu_q=base.dcu, max_q=rows,
                            out=out, lse=lse, workspace=ws)

    cache = (base.dk.view(torch.uint8), base.dv.view(torch.uint8), base.dks, base.dvs)
    start = [t.clone() for t in cache]

    def place(new, ctx):
        for t, s in zip(cache, start):
            t.copy_(s)
        base.dcu.copy_(torch.tensor([0, new[0], new[0] + new[1], sum(new)], dtype=torch.int32))
        base.dctx.copy_(torch.tensor(ctx, dtype=torch.int32))
        out.fill_(7.0)
        lse.fill_(7.0)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new, ctx in steps + steps[::-1]:
        place(new, ctx)
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (out, lse, *cache)]
        place(new, ctx)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for t, w in zip((out, lse, *cache), want))


def test_two_graphs_share_a_workspace(P):  # noqa: F811
    """Two captured calls with one workspace, replayed in turn on a stream."""
    cases = [Case(270 + i, "fp16", new, ctx, 8, 2, 128, 64)
             for i, (new, ctx) in enumerate((([1, 2], [6000, 900]), ([5, 1, 9], [3000, 8000, 100])))]
    qs, need = [], 0
    for c in cases:
        c.upload()
        qs.append(c.act(8).to(DEV))
        need = max(need, P.awq_attn_kv8_workspace_size(len(c.new), c.rows, 8, 2, 128, 64, c.bt.shape[1], max(c.new)))
    assert need > 0
    want = [run_attn(P, c, q, max_q=max(c.new)) for c, q in zip(cases, qs)]
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    outs, graphs = [torch.zeros_like(q) for q in qs], []
    for c, q, o in zip(cases, qs, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            P.awq_attn_kv8(q, c.dk, c.dv, c.dks, c.dvs, c.dbt, c.dctx, cu_q=c.dcu, max_q=max(c.new), out=o, workspace=ws)
        graphs.append(graph)
    for _ in range(4):
        for o in outs:
            o.fill_(7.0)
        for graph in graphs:
            graph.replay()
        for o, w in zip(outs, want):
            assert torch.equal(o, w[0])
