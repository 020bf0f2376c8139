"""Linears with an epilogue, routing, products grouped by expert and their combination, against
float64 (tests/moe_ref.py)."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from tests import moe_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def P():
    import weight_only_int4_awq_amd as P
    P.load()
    return P


def gen(seed):
    return torch.Generator().manual_seed(seed)


def tokens(g, rows, k, dt):
    x = torch.randn(rows, k, generator=g) * (1 + 9 * (torch.rand(k, generator=g) < 0.02))
    # bf16 activations within fp16's normal range: values below it lose bits by contract
    x = torch.where(x.abs() < 2.0 ** -10, torch.full_like(x, 2.0 ** -10), x)
    return x.to(dt)


def guarded(rows, n, dt, pad=64):
    """An output between two runs of a sentinel, and a check that they are whole."""
    whole = torch.full((rows * n + 2 * pad,), 77.0, dtype=dt, device=DEV)
    return whole[pad:pad + rows * n].view(rows, n), lambda: bool((whole[:pad] == 77).all() and (whole[-pad:] == 77).all())


def dense(P, m, n, k, g, dt, act="none", gated=False, bias=False, inv=False, residual=False, seed=0):
    ge = gen(seed + 1000 * m + n + 7 * k + g)
    nw = 2 * n if gated else n
    qw, sc, qz = R.packed(ge, (), nw, k, g)
    x = tokens(ge, m, k, dt)
    b = torch.randn(nw, generator=ge).to(dt) if bias else None
    iv = torch.exp(0.4 * torch.randn(k, generator=ge)).half() if inv else None
    r = (3 * torch.randn(m, n, generator=ge)).to(dt) if residual else None
    d = lambda t: None if t is None else t.to(DEV)
    out, whole = guarded(m, n, dt)
    need = P.awq_linear_act_workspace_size(m, n, k, g, gated, inv, dt is BF16)
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    fn = P.awq_linear_w4a16_act_bf16 if dt is BF16 else P.awq_linear_w4a16_act
    args = (d(x), d(qw), d(sc), d(qz), d(iv), d(b), act, gated, d(r), g)
    y = fn(*args, out=out, workspace=ws[:need])
    again = fn(*args)
    assert y.data_ptr() == out.data_ptr() and whole() and bool((ws[need:] == 0xA5).all())
    assert torch.equal(y, again)
    v, bound = R.linear(x, R.weights(qw, sc, qz, g), iv, b, act, gated, r, dt)
    R.check(y, v, bound, (m, n, k, g, dt, act, gated, bias, inv, residual))


@pytest.mark.parametrize("m", [1, 2, 7, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 127, 128, 129, 200, 257, 513])
@pytest.mark.parametrize("n,k,g", [(1, 64, 32), (33, 192, 64), (130, 384, 128), (264, 1088, 64)])
def test_dense_rows_and_odd_sizes(P, m, n, k, g):
    for i, dt in enumerate((F16, BF16)):
        dense(P, m, n, k, g, dt, seed=i)


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m", [1, 5, 20, 40, 130, 300])
def test_dense_epilogues(P, m, act, gated):
    i = 0
    for bias in (False, True):
        for inv in (False, True):
            for residual in (False, True):
                i += 1
                n, k, g = [(72, 256, 128), (45, 320, 64), (136, 96 * 2, 32)][i % 3]
                dense(P, m, n, k, g, (F16, BF16)[i // 2 % 2], act, gated, bias, inv, residual, seed=i)


@pytest.mark.parametrize("m,n,k,g,gated", [(1, 1024, 4096, 128, True), (4, 4096, 1024, 128, False),
                                           (17, 1024, 8192, 128, False), (40, 512, 14336, 128, False),
                                           (100, 640, 4096, 64, True), (1, 64, 14336, 32, False),
                                           (333, 4099, 1088, 64, False), (640, 2048, 2048, 128, True)])
def test_dense_longer(P, m, n, k, g, gated):
    dense(P, m, n, k, g, F16, "silu" if gated else "none", gated, True, True, True)
    dense(P, m, n, k, g, BF16, "silu" if gated else "none", gated)


# every form of the tiles: rows, K-step, K groups, K slices, with odd numbers of groups and ragged ends
@pytest.mark.parametrize("m,n,k,g,gated", [(600, 2000, 128, 64, False), (600, 2040, 192, 64, False), (600, 1000, 160 * 2, 32, True),
                                           (2000, 4090, 64, 64, False), (2000, 4096, 128, 128, False), (2000, 2050, 64, 32, True),
                                           (640, 4096, 1024, 128, False), (640, 2048, 1088, 64, True), (640, 4000, 960, 32, False),
                                           (1500, 8192, 320, 64, False), (1500, 4096, 384, 128, True), (1500, 8200, 320, 32, False),
                                           (640, 4096, 2688, 128, False), (640, 4096, 2752, 64, False), (640, 2048, 2720 - 32, 32, True),
                                           (1100, 8192, 1408, 128, False), (1100, 4100, 1984, 64, True), (1100, 8192, 1472, 32, False),
                                           (24, 16384, 4096, 128, False), (24, 8192, 4160, 64, True), (24, 16384, 4096, 32, False),
                                           (40, 8192, 4096, 128, False), (50, 4096, 4160, 64, True), (40, 8192, 4096, 32, False),
                                           (200, 4096, 4224, 128, True), (200, 8192, 4160, 64, False), (200, 8192, 4096, 32, False)])
def test_dense_tiles(P, m, n, k, g, gated):
    i = m + n + k
    dense(P, m, n, k, g, (F16, BF16)[i // 64 % 2], ("none", "silu")[gated], gated, bool(i // 32 % 2), bool(i // 128 % 2), not gated)


@pytest.mark.parametrize("m,n,k,g,gated", [(600, 1000, 1024, 128, False), (530, 260, 960, 32, True), (600, 2040, 4096, 64, False),
                                            (600, 2040, 8192, 128, False), (513, 1000, 7104, 64, True)])
def test_dense_split_beyond_512_rows(P, m, n, k, g, gated):
    """Matrices of few tiles, split along K: tiles of 32, 64 and 128 rows."""
    dense(P, m, n, k, g, BF16 if gated else F16, "gelu" if gated else "none", gated, True, True, True)


def test_dense_extremes(P):
    """Activations at their ends, scales of zero and NaN, inputs with inf and NaN: as in float64, and only where they belong."""
    k, n, g = 128, 40, 128
    ge = gen(5)
    for m in (3, 40, 140):
        qw, sc, qz = R.packed(ge, (), n, k, g, scale=3.0)
        x = tokens(ge, m, k, F16)
        sc[5], sc[6] = 0.0, math.nan
        x[1, 7], x[2, 9] = math.inf, math.nan
        w = R.weights(qw, sc, qz, g)
        for act in R.ACTS[1:]:
            y = P.awq_linear_w4a16_act(x.to(DEV), qw.to(DEV), sc.to(DEV), qz.to(DEV), act=act, g=g).cpu()
            assert y[:, 6].isnan().all() and y[2].isnan().all()
            rest = [i for i in range(m) if i not in (1, 2)]
            cols = [i for i in range(n) if i != 6]
            v, b = R.linear(x[rest], w[cols], None, None, act, False, None, F16)
            big = v.abs() > 65504                                      # beyond fp16: inf
            got = y[rest][:, cols]
            R.check(torch.where(big, v.half(), got), torch.where(big, v.half().double(), v), torch.where(big, torch.zeros_like(b), b).nan_to_num(0), act)
            assert bool((got[v.abs() > 70000].isinf()).all())
            assert bool((got[:, 5] == 0).all())


@pytest.mark.parametrize("rows", [1, 3, 4])
@pytest.mark.parametrize("k,g", [(1024, 128), (1152, 128), (1024, 64), (320, 64), (1024, 32), (96 * 2, 32)])
def test_few_rows_keep_the_product_with_the_inverse_scale(P, rows, k, g):
    """Even channels give (1 + 2^-10)^2, odd ones -(1 + 2^-9): equal once rounded to fp16, 2^-20 apart.

    Sums of the rounded products are multiples of 2^-9 below 2^13 and those of what was lost multiples of
    2^-20 below 1, row by row times a power of two: exact in any order, and so is the result."""
    n, e = 33, 3
    x, inv = torch.full((rows, k), 1 + 2.0 ** -9), torch.ones(k)
    x[:, ::2], inv[::2] = 1 + 2.0 ** -10, 1 + 2.0 ** -10
    x *= 2.0 ** torch.arange(rows)[:, None]                            # rows apart from each other
    x, inv = x.half().to(DEV), inv.half().to(DEV)
    qw = torch.full((e, n, k // 8), 0x79797979, dtype=torch.int32, device=DEV)      # q - z = 1, -1, 1 ..
    sc = torch.ones(e, n, k // g, dtype=torch.float16, device=DEV)
    zeros = torch.zeros(e, n, (k // g + 7) // 8 * 8, dtype=torch.int64)
    zeros[..., :k // g] = 8
    words = sum(zeros[..., j::8] << (4 * j) for j in range(8))
    qz = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int().to(DEV)
    want = (k * 2.0 ** -21 * 2.0 ** torch.arange(rows, dtype=torch.float64))[:, None].expand(rows, n)
    y = P.awq_linear_w4a16_act(x, qw[0], sc[0], qz[0], inv, g=g)
    assert torch.equal(y.cpu().double(), want)
    offsets = torch.tensor([0, 0, rows, rows], dtype=torch.int32, device=DEV)
    y = P.awq_moe_linear_w4a16(x, qw, sc, qz, offsets, inv_s16=inv, g=g)
    assert torch.equal(y.cpu().double(), want)


def test_few_rows_whose_product_leaves_the_range(P):
    """x inv_s beyond fp16 is infinite, with its sign, for its own row alone."""
    k, n = 256, 17
    x = torch.ones(4, k)
    x[1, 3], x[2, 200] = 60000, -60000
    qw = torch.full((n, k // 8), -0x66666667, dtype=torch.int32, device=DEV)        # q = 9
    sc, qz = torch.full((n, 2), 0.25).half().to(DEV), torch.full((n, 1), 0x88, dtype=torch.int32, device=DEV)
    y = P.awq_linear_w4a16_act(x.half().to(DEV), qw, sc, qz, torch.full((k,), 2.0).half().to(DEV)).cpu()
    assert (y[1] == math.inf).all() and (y[2] == -math.inf).all() and (y[[0, 3]] == 128).all()


# ---------------------------------------------------------------- routing

def check_route(P, logits, topk, scoring, renorm, scale):
    t, e = logits.shape
    out = (torch.full((t, topk), -7, dtype=torch.int32, device=DEV), torch.full((t, topk), -7.0, device=DEV),
           torch.full((e + 1,), -7, dtype=torch.int32, device=DEV), torch.full((t * topk,), -7, dtype=torch.int32, device=DEV),
           torch.full((t, topk), -7, dtype=torch.int32, device=DEV))
    got = P.awq_moe_route(logits.to(DEV), topk, scoring, renorm, scale, out=out)
    want = R.route(logits, topk, scoring, renorm, scale)
    for name, a, b in zip(("ids", "weights", "offsets", "row_slot", "slot_row"), got, want):
        if name != "weights":
            assert torch.equal(a.cpu(), b), (name, t, e, topk)
    w, v = got[1].double().cpu(), want[1]
    assert torch.equal(w.isnan(), v.isnan())
    # exp within 2 ulp of an argument rounded once (2^-24 |x - max|, up to 90), sums of up to e terms, three quotients
    assert bool(((w - v).abs() <= (e + 120) * 2.0 ** -24 * v.abs() + 1e-37).logical_or(v.isnan()).all()), (t, e, topk)
    again = P.awq_moe_route(logits.to(DEV), topk, scoring, renorm, scale)
    n = int(got[2][-1])
    assert all(torch.equal(a.nan_to_num(9.0) if a.is_floating_point() else a[:n] if i == 3 else a,
                           b.nan_to_num(9.0) if b.is_floating_point() else b[:n] if i == 3 else b)
               for i, (a, b) in enumerate(zip(got, again)))


@pytest.mark.parametrize("t", [0, 1, 2, 15, 63, 64, 65, 130, 1000])
@pytest.mark.parametrize("e,topk", [(1, 1), (2, 2), (8, 2), (60, 4), (64, 8), (65, 3), (128, 8), (257, 6), (1024, 32)])
def test_route(P, t, e, topk):
    ge = gen(t + 3 * e)
    i = t + e
    dt = (torch.float32, F16, BF16)[i % 3]
    x = (2 * torch.randn(t, e, generator=ge)).to(dt)
    check_route(P, x, topk, ("softmax", "sigmoid")[i % 2], bool(i // 2 % 2), (1.0, 2.5)[i // 3 % 2])
    # ties, zeros of both signs, closed experts, padded tokens, NaN and infinities
    y = torch.randint(-2, 3, (t, e), generator=ge).to(dt)
    y = torch.where(torch.rand(t, e, generator=ge) < 0.3, torch.full_like(y, -math.inf), y)
    y = torch.where(torch.rand(t, e, generator=ge) < 0.1, torch.full_like(y, -0.0), y)
    if t > 10:
        y[3] = -math.inf
        y[5, e // 2] = math.nan
        y[6] = math.nan
        y[7, e - 1] = math.inf
        y[t - 4:] = -math.inf
    for scoring in ("softmax", "sigmoid"):
        for renorm in (False, True):
            check_route(P, y, topk, scoring, renorm, 1.5)


@pytest.mark.parametrize("dt", [torch.float32, F16, BF16])
@pytest.mark.parametrize("e,topk", [(1, 1), (7, 3), (8, 8), (16, 16), (24, 5), (63, 16), (100, 16), (100, 17), (120, 2), (128, 16), (128, 32), (129, 4),
                                    (200, 8), (256, 16), (256, 17), (257, 3), (400, 8), (511, 5), (512, 16)])
def test_route_four_tokens_to_a_wave(P, dt, e, topk):
    """Many tokens of up to 512 experts: whole and part rows of lanes, both widths of loads, ties, closed and NaN."""
    ge = gen(e + topk)
    for t, away in ((49, 0), (77, 1), (200, 0)):
        x = torch.randint(-6, 7, (t, e), generator=ge).to(dt) / 2                      # many ties
        x[torch.rand(t, e, generator=ge) < 0.3] = -math.inf
        x[3], x[t - 1] = -math.inf, math.nan
        x[5, e // 2] = math.nan
        x[7, e - 1] = 40.0
        flat = torch.zeros(t * e + away, dtype=dt, device=DEV)                         # one element past 16 bytes
        flat[away:] = x.to(DEV).flatten()
        for i, scoring in enumerate(("softmax", "softmax", "sigmoid", "sigmoid")):
            check_route(P, flat[away:].view(t, e), topk, scoring, bool(i & 1), 1.5)


def test_route_many(P):
    """More tokens than work-groups hold at 64 each: chunks of several rounds, every expert of one popular."""
    ge = gen(2)
    x = torch.randn(20011, 16, generator=ge)
    x[:, 3] += 4
    got = P.awq_moe_route(x.to(DEV), 3)
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :3].int()
    assert torch.equal(got[0].cpu(), ids)
    flat = ids.flatten().long()
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(got[3].cpu().long(), order)
    assert torch.equal(got[2].cpu().long(), torch.cat((torch.zeros(1, dtype=torch.int64), torch.bincount(flat, minlength=16).cumsum(0))))
    assert torch.equal(got[4].cpu().flatten().long()[order], torch.arange(len(flat)))


def test_route_extreme_logits(P):
    """Logits at the ends of their type, and sigmoids that underflow."""
    big = torch.tensor([[3e38, -3e38, 1e38, 0.0], [-3e38, -3.2e38, -1e38, -2e38], [200.0, 199.0, -200.0, 0.0],
                        [-150.0, -200.0, -160.0, -170.0]])
    for renorm in (False, True):
        check_route(P, big[:3], 3, "softmax", renorm, 1.0)
    got = P.awq_moe_route(big.to(DEV), 2, "sigmoid", True)
    assert got[0].cpu().tolist() == [[0, 2], [2, 3], [0, 1], [0, 2]]
    assert got[1].cpu().tolist()[1] == [0.0, 0.0] and got[1].cpu().tolist()[3] == [0.0, 0.0]


# ---------------------------------------------------------------- products grouped by expert

def split(e, counts):
    return torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)


def grouped(P, counts, n, k, g, dt, gather, act="none", gated=False, bias=False, inv=False, topk=2, behind=3, seed=0):
    e = len(counts)
    ge = gen(seed + sum(counts) + n + k)
    nw = 2 * n if gated else n
    qw, sc, qz = R.packed(ge, (e,), nw, k, g)
    offsets = split(e, counts)
    used = int(offsets[-1])
    rows = used + behind
    t = max(1, (rows + topk - 1) // topk)
    row_slot = torch.randint(0, t * topk, (rows,), generator=ge).int() if gather else None     # some of them twice
    x = tokens(ge, t if gather else rows, k, dt)
    b = torch.randn(e, nw, generator=ge).to(dt) if bias else None
    iv = torch.exp(0.4 * torch.randn(k, generator=ge)).half() if inv else None
    d = lambda v: None if v is None else v.to(DEV)
    out, whole = guarded(rows, n, dt)
    out.fill_(-5)
    need = P.awq_moe_linear_workspace_size(rows, x.shape[0], e, n, k, g, gated, inv, dt is BF16)
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    fn = P.awq_moe_linear_w4a16_bf16 if dt is BF16 else P.awq_moe_linear_w4a16
    y = fn(d(x), d(qw), d(sc), d(qz), d(offsets), d(row_slot), topk, d(iv), d(b), act, gated, g, out=out,
           workspace=ws[:need])
    assert whole() and bool((ws[need:] == 0xA5).all()) and bool((y[used:] == -5).all())
    y = y.cpu()
    for j in range(e):
        a, z = int(offsets[j]), int(offsets[j + 1])
        if a < z:
            src = x[row_slot[a:z].long() // topk] if gather else x[a:z]
            v, bound = R.linear(src, R.weights(qw[j], sc[j], qz[j], g), iv, None if b is None else b[j], act, gated,
                                None, dt)
            R.check(y[a:z], v, bound, (j, counts, n, k, g, dt, gather, act, gated))


COUNTS = [[1], [0, 3, 0], [16, 17, 1, 0, 33], [0, 0, 0, 0, 0, 5], [2] * 20, [130, 0, 1], [64, 65, 63, 128, 129],
          [300, 2, 90, 0, 200], [1, 0] * 50, [20] * 70 + [0, 90]]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(P, counts, gather):
    grouped(P, counts, 72, 256, 128, F16, gather, "silu", True, True, False)
    grouped(P, counts, 33, 192, 64, BF16, gather, "none", False, True, True)
    grouped(P, counts, 264, 64, 32, F16, gather, "gelu", False, False, True, topk=3)
    grouped(P, counts, 24, 320, 64, BF16, gather, "gelu_tanh", True, False, False, topk=1)


@pytest.mark.parametrize("e,most", [(1024, 4), (129, 30), (200, 90)])
def test_grouped_many_experts(P, e, most):
    g = gen(3)
    counts = torch.randint(0, most, (e,), generator=g).tolist()
    grouped(P, counts, 16, 64, 64, F16, True, "silu", True)
    grouped(P, counts, 40, 128, 128, BF16, False, "none", False, True, True)


@pytest.mark.parametrize("bad", [[0, -3, 2, 9], [5, 1, 0, 4], [0, 4, 1000000, 2000000000], [-2 ** 31, 2 ** 31 - 1, -1, 3],
                                 [0, 9, 9, 8], [-1, 2, 3, 4]])
@pytest.mark.parametrize("rows", [9, 150])
def test_grouped_plans_out_of_order_write_nothing(P, bad, rows):
    e, n, k = 3, 40, 128
    ge = gen(1)
    qw, sc, qz = (t.to(DEV) for t in R.packed(ge, (e,), n, k, 128))
    x = tokens(ge, 4, k, F16).to(DEV)
    slots = torch.arange(rows, dtype=torch.int32, device=DEV) % 8
    out, whole = guarded(rows, n, F16)
    out.fill_(-5)
    P.awq_moe_linear_w4a16(x, qw, sc, qz, torch.tensor(bad, dtype=torch.int32, device=DEV), slots, 2, out=out)
    torch.cuda.synchronize()
    assert whole() and bool((out == -5).all())
    many = torch.zeros(1025, dtype=torch.int32)                                  # the bad one among many experts
    many[700:] = rows
    many[900] = rows + 1
    qw, sc, qz = (t[:1].repeat(1024, 1, 1).contiguous() for t in (qw, sc, qz))
    P.awq_moe_linear_w4a16(x, qw, sc, qz, many.to(DEV), slots, 2, out=out)
    torch.cuda.synchronize()
    assert whole() and bool((out == -5).all())


@pytest.mark.parametrize("bad", [[0, 3, 3, 9], [2, 2, 8, 9]])
@pytest.mark.parametrize("rows", [9, 150])
def test_grouped_any_slots_stay_inside(P, bad, rows):
    """Slots of any value: nothing outside the tensors is read or written, and the call returns."""
    e, n, k = 3, 40, 128
    ge = gen(1)
    qw, sc, qz = (t.to(DEV) for t in R.packed(ge, (e,), n, k, 128))
    x = tokens(ge, 4, k, F16).to(DEV)
    slots = torch.tensor([2 ** 31 - 1, -5, 7, 0, 3, -2 ** 31, 100, 8, 1] * 17, dtype=torch.int32)[:rows].to(DEV)
    out, whole = guarded(rows, n, F16)
    out.fill_(-5)
    P.awq_moe_linear_w4a16(x, qw, sc, qz, torch.tensor(bad, dtype=torch.int32, device=DEV), slots, 2, out=out)
    torch.cuda.synchronize()
    assert whole() and bool((out[:bad[0]] == -5).all() and (out[bad[-1]:] == -5).all() and out[bad[0]:bad[-1]].isfinite().all())


@pytest.mark.parametrize("topk", [1, 3, 4, 32])
@pytest.mark.parametrize("rows", [12, 300])
def test_far_slots(P, topk, rows):
    """Tokens up to the last of an x of nearly 4 GiB, slots up to 2^27."""
    k, n, g = 64, 48, 64
    t = min((1 << 31) // k - 1, (1 << 27) // topk)
    ge = gen(topk)
    p = R.packed(ge, (2,), n, k, g)
    x = torch.empty(t, k, dtype=F16, device=DEV)
    far = torch.unique(torch.cat((torch.arange(t - rows // 2, t), torch.randint(0, t, (rows,), generator=ge))))[-rows:]
    slots = (far * topk + torch.randint(0, topk, far.shape, generator=ge)).int()
    xs = tokens(ge, len(far), k, F16)
    x[far.to(DEV)] = xs.to(DEV)
    r = len(far)
    y = P.awq_moe_linear_w4a16(x, *(q.to(DEV) for q in p), torch.tensor([0, r // 3, r], dtype=torch.int32, device=DEV),
                               slots.to(DEV), topk, g=g).cpu()
    for j, (a, z) in enumerate(((0, r // 3), (r // 3, r))):
        v, bound = R.linear(xs[a:z], R.weights(*(q[j] for q in p), g), None, None, "none", False, None, F16)
        R.check(y[a:z], v, bound, (topk, j))


# ---------------------------------------------------------------- combination

@pytest.mark.parametrize("t,n,topk", [(1, 8, 1), (3, 5, 2), (64, 2048, 8), (7, 1001, 9), (130, 264, 32), (0, 16, 2)])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_combine(P, t, n, topk, dt):
    ge = gen(t + n)
    r = t * topk + 2
    rows = torch.randn(r, n, generator=ge).to(dt)
    w = torch.rand(t, topk, generator=ge)
    sr = torch.randint(0, r, (t, topk), generator=ge).int()                     # some rows twice
    gone = torch.rand(t, topk, generator=ge) < 0.2
    sr = torch.where(gone, torch.full_like(sr, -1), sr)
    for res in (None, (2 * torch.randn(t, n, generator=ge)).to(dt)):
        out, whole = guarded(t, n, dt)
        fn = P.awq_moe_combine_bf16 if dt is BF16 else P.awq_moe_combine
        y = fn(rows.to(DEV), w.to(DEV), sr.to(DEV), None if res is None else res.to(DEV), out=out)
        part = torch.where(gone[..., None], torch.zeros(1, dtype=torch.float64), rows[sr.clamp(min=0).long()].double() * w[..., None].double())
        v, mag = part.sum(1), part.abs().sum(1)
        if res is not None:
            v, mag = v + res.double(), mag + res.double().abs()
        R.check(y, v, (topk + 1) * 2.0 ** -24 * mag + R.HALF[dt] * 1.001 * v.abs() + 2.0 ** -25, (t, n, topk))
        assert whole()
        if res is not None:                                                     # in place
            rd = res.to(DEV)
            assert torch.equal(fn(rows.to(DEV), w.to(DEV), sr.to(DEV), rd, out=rd), y)


def test_combine_without_rows_and_with_nan(P):
    rows = torch.full((2, 16), math.inf, dtype=F16, device=DEV)
    w = torch.tensor([[0.0, 0.0], [math.nan, math.nan], [1.0, 0.5]], device=DEV)
    sr = torch.tensor([[-1, -1], [-1, -1], [2, -2 ** 31]], dtype=torch.int32, device=DEV)
    y = P.awq_moe_combine(rows, w, sr).cpu()
    assert bool((y[0] == 0).all() and y[1].isnan().all() and (y[2] == 0).all())
    none = P.awq_moe_combine(rows[:0], w[:1], sr[:1], residual=torch.ones(1, 16, dtype=F16, device=DEV))
    assert bool((none == 1).all())


# ---------------------------------------------------------------- together

def block(P, x, logits, gate_up, down, topk, dt, ws=None):
    """A mixture-of-experts block as a decoder layer runs it."""
    bf = dt is BF16
    up = P.awq_moe_linear_w4a16_bf16 if bf else P.awq_moe_linear_w4a16
    add = P.awq_moe_combine_bf16 if bf else P.awq_moe_combine
    _, w, offsets, row_slot, slot_row = P.awq_moe_route(logits, topk)
    h = up(x, *gate_up, offsets, row_slot, topk, act="silu", gated=True)
    y = up(h, *down, offsets)
    return add(y, w, slot_row, residual=x)


def block_ref(x, logits, gate_up, down, topk, dt):
    """(value, bound): h is rounded to the activation type between the two projections."""
    ids, w, _, _, _ = R.route(logits, topk, "softmax", True, 1.0)
    v, bound = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    for j in range(gate_up[0].shape[0]):
        tok, choice = (ids == j).nonzero(as_tuple=True)
        if len(tok):
            h, dh = R.linear(x[tok], R.weights(*(p[j] for p in gate_up), 128), None, None, "silu", True, None, dt)
            wd = R.weights(*(p[j] for p in down), 128)
            y, dy = R.linear(h.to(dt), wd, None, None, "none", False, None, dt)
            y = h @ wd.t()
            dy = dy * 1.02 + 2 * (dh + R.HALF[dt] * h.abs()) @ wd.abs().t()
            c = w[tok, choice][:, None]
            v.index_add_(0, tok, c * y)
            bound.index_add_(0, tok, c * dy + 1e-5 * (c * y).abs())
    return v, bound + R.HALF[dt] * 1.01 * (v.abs() + bound)


@pytest.mark.parametrize("t,e,topk,dt", [(1, 8, 2, F16), (9, 16, 4, BF16), (70, 4, 2, F16), (300, 6, 3, BF16)])
def test_block(P, t, e, topk, dt):
    ge = gen(t)
    k, n = 256, 384
    gate_up, down = R.packed(ge, (e,), 2 * n, k, 128), R.packed(ge, (e,), k, n, 128)
    x = tokens(ge, t, k, dt)
    logits = torch.randn(t, e, generator=ge)
    logits[:, e - 1] = -math.inf
    if t > 20:
        logits[t - 5:] = -math.inf                                              # padded tokens keep their residual
    up = lambda p: tuple(q.to(DEV) for q in p)
    y = block(P, x.to(DEV), logits.to(DEV), up(gate_up), up(down), topk, dt)
    v, bound = block_ref(x, logits, gate_up, down, topk, dt)
    R.check(y, v, bound, (t, e))
    if t > 20:
        assert torch.equal(y[t - 5:].cpu(), x[t - 5:])


@pytest.mark.parametrize("t", [3, 90])
def test_block_captured_and_replayed_with_other_routing(P, t):
    ge = gen(t)
    e, topk, k, n = 8, 2, 256, 256
    gate_up = tuple(q.to(DEV) for q in R.packed(ge, (e,), 2 * n, k, 128))
    down = tuple(q.to(DEV) for q in R.packed(ge, (e,), k, n, 128))
    x, logits = torch.zeros(t, k, dtype=F16, device=DEV), torch.zeros(t, e, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block(P, x, logits, gate_up, down, topk, F16)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(P, x, logits, gate_up, down, topk, F16)
    for i in range(4):
        xi, li = tokens(ge, t, k, F16), torch.randn(t, e, generator=ge)
        if i == 2:
            li[:, 1:] = -math.inf                                               # every token to one expert
        x.copy_(xi)
        logits.copy_(li)
        graph.replay()
        got = y.clone()
        assert torch.equal(got, block(P, xi.to(DEV), li.to(DEV), gate_up, down, topk, F16)), i
        torch.cuda.synchronize()


def test_two_streams(P):
    """Two calls at once, each with its own workspace, bit for bit what each gives alone."""
    ge = gen(4)
    k, n, m = 1024, 512, 100
    p = tuple(q.to(DEV) for q in R.packed(ge, (), n, k, 128))
    xs = [tokens(ge, m, k, BF16).to(DEV) for _ in range(2)]
    alone = [P.awq_linear_w4a16_act_bf16(x, *p, act="gelu") for x in xs]
    logits = [torch.randn(500, 32, generator=ge).to(DEV) for _ in range(2)]
    routed = [P.awq_moe_route(v, 4) for v in logits]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        outs = []
        for s, x, v in zip(streams, xs, logits):
            with torch.cuda.stream(s):
                outs.append((P.awq_linear_w4a16_act_bf16(x, *p, act="gelu"), P.awq_moe_route(v, 4)))
        torch.cuda.synchronize()
        for (y, r), a, ra in zip(outs, alone, routed):
            assert torch.equal(y, a) and all(torch.equal(u, w) for u, w in zip(r, ra))


@pytest.mark.parametrize("t", [2, 120])
def test_two_threads(P, t):
    """The whole layer from two threads at once, a stream each, with the binding's own workspaces."""
    import threading
    ge = gen(40 + t)
    e, topk, k, n = 6, 2, 256, 384
    gate_up = tuple(q.to(DEV) for q in R.packed(ge, (e,), 2 * n, k, 128))
    down = tuple(q.to(DEV) for q in R.packed(ge, (e,), k, n, 128))
    xs = [tokens(ge, t, k, BF16).to(DEV) for _ in range(2)]
    logits = [torch.randn(t, e, generator=ge).to(DEV) for _ in range(2)]
    want = [block(P, x, v, gate_up, down, topk, BF16) for x, v in zip(xs, logits)]
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    got[i].append(block(P, xs[i], logits[i], gate_up, down, topk, BF16))
            s.synchronize()
        except BaseException as err:                  # noqa: BLE001
            failed.append(err)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failed, failed
    for ys, w in zip(got, want):
        assert len(ys) == 20 and all(torch.equal(y, w) for y in ys)


def test_two_graphs_with_one_workspace(P):
    """Captured with the same scratch and replayed in turn on one stream: each what it gives alone."""
    ge = gen(50)
    m, k, n, e = 100, 512, 768, 40
    p = tuple(q.to(DEV) for q in R.packed(ge, (), n, k, 128))
    inv = torch.exp(0.4 * torch.randn(k, generator=ge)).half().to(DEV)
    ws = torch.zeros(max(P.awq_linear_act_workspace_size(m, n, k, 128, False, True, True),
                         P.awq_moe_route_workspace_size(m, e)), dtype=torch.uint8, device=DEV)
    xs = [torch.zeros(m, k, dtype=BF16, device=DEV) for _ in range(2)]
    logits = [torch.zeros(m, e, device=DEV) for _ in range(2)]

    def step(x, v, ws):
        return (P.awq_linear_w4a16_act_bf16(x, *p, inv, act="silu", workspace=ws), *P.awq_moe_route(v, 4, workspace=ws))

    step(xs[0], logits[0], ws)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, v in zip(xs, logits):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(x, v, ws))
        graphs.append(graph)
    for _ in range(4):
        for x, v in zip(xs, logits):
            x.copy_(tokens(ge, m, k, BF16))
            v.copy_(torch.randn(m, e, generator=ge))
        for graph in graphs:
            graph.replay()
        for out, x, v in zip(outs, xs, logits):
            assert all(torch.equal(a, b) for a, b in zip(out, step(x, v, None)))
        torch.cuda.synchronize()


def test_residual_in_place_and_far_offsets(P):
    """residual is out; and rows of y and x beyond 2^31 elements of a tensor."""
    ge = gen(6)
    k, n = 128, 256
    p = tuple(q.to(DEV) for q in R.packed(ge, (), n, k, 128))
    for m in (5, 40, 200):
        x = tokens(ge, m, k, F16).to(DEV)
        r = torch.randn(m, n, generator=ge).half().to(DEV)
        y = P.awq_linear_w4a16_act(x, *p, residual=r)
        assert torch.equal(P.awq_linear_w4a16_act(x, *p, residual=r, out=r), y)
    rows = (1 << 31) // n + 40                                                  # y: 4 GiB and more
    x = tokens(ge, 64, k, F16).to(DEV)
    e = 2
    pe = tuple(torch.stack((q, q)) for q in p)
    slots = (torch.arange(rows, device=DEV, dtype=torch.int32) % 64)
    offsets = torch.tensor([0, rows - 40, rows], dtype=torch.int32, device=DEV)
    y = P.awq_moe_linear_w4a16(x, *pe, offsets, slots, 1)
    want = P.awq_linear_w4a16_act(x, *p)
    for a in (0, rows // 2, rows - 100):
        got = y[a:a + 100]
        ref = want[slots[a:a + 100].long()]
        assert bool(((got.float() - ref.float()).abs() <= 4 * R.HALF[F16] * ref.float().abs().amax()).all()), a
