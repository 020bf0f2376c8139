"""Edges of the linears with an epilogue, of products grouped by expert and of their combination,
against float64 (tests/moe_ref.py) or to the bit."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from tests import moe_ref as R  # noqa: E402
from tests.test_gpu_moe import grouped  # noqa: E402

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


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("k,g", [(512, 128), (1152, 128), (320, 64), (192, 32)])
def test_a_row_among_its_expert(P, k, g, dt):
    """One token in every row: every row of an expert has the same bits, whatever tile it fell in, and
    experts of up to four rows have those of the dense call."""
    ge = gen(k + g)
    n, counts = 40, [9, 1, 12, 3, 4, 5, 8, 17, 0, 2]
    e, rows = len(counts), sum(counts)
    qw, sc, qz = (t.repeat(e, 1, 1).to(DEV) for t in R.packed(ge, (1,), n, k, g))
    inv = torch.exp(0.4 * torch.randn(k, generator=ge)).half().to(DEV)
    x = torch.randn(1, k, generator=ge).to(dt).to(DEV)
    offsets = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    slots = torch.zeros(rows + 3, dtype=torch.int32, device=DEV)
    dense, grouped = ((P.awq_linear_w4a16_act_bf16, P.awq_moe_linear_w4a16_bf16) if dt is BF16 else
                      (P.awq_linear_w4a16_act, P.awq_moe_linear_w4a16))
    assert rows + 3 > 6 * e                                             # tiles
    y = grouped(x, qw, sc, qz, offsets, slots, 1, inv_s16=inv, g=g)[:rows]
    assert bool((y == y[:1]).all())
    more = e + 9                                                        # streams: fewer rows to an expert on average
    qw, sc, qz = (t[:1].repeat(more, 1, 1) for t in (qw, sc, qz))
    ends = torch.cat((offsets, offsets[-1:].repeat(9)))
    y = grouped(x, qw, sc, qz, ends, slots[:rows], 1, inv_s16=inv, g=g)
    at = ends.tolist()
    few = dense(x, qw[0], sc[0], qz[0], inv, g=g)[0]
    many = y[at[counts.index(9)]]
    for j, c in enumerate(counts):
        mine = y[at[j]:at[j + 1]]
        assert bool((mine == (few if c <= 4 else many)).all()), (j, c)


# by tiles of 32, 64 and 128 rows, with two K groups, K slices and neither
TILES = [(m, n, k, g) for m, n, k in ((700, 2050, 768), (2000, 4096, 192), (2000, 4096, 768), (2100, 8192, 768),
                                      (1100, 8192, 512), (1000, 2048, 1536), (640, 4096, 1920)) for g in (128, 64, 32)]
# streaming with 8 and 16 rows
STREAMS = [(m, n, k, g) for m, n, k in ((1, 48, 384), (4, 48, 512), (8, 72, 320), (16, 40, 512), (40, 40, 384),
                                        (300, 520, 448), (300, 2050, 512)) for g in (128, 64, 32)]


def scattered_scales(ge, n, ng):
    """Scales of all mantissas over 2^-10 .. 2^-1, every seventh of them zero, and a row of zeros."""
    sc = (2.0 ** (-1 - 9 * torch.rand(n, ng, generator=ge))).half()
    sc[torch.rand(n, ng, generator=ge) < 1 / 7] = 0
    sc[3] = 0
    return sc


@pytest.mark.parametrize("m,n,k,g", TILES + STREAMS)
@pytest.mark.parametrize("dt", [F16, BF16])
def test_weights_enter_exactly(P, m, n, k, g, dt):
    """Codes of one value in every group times a scale that leaves no code but 0, 1, 2, 4 and 8 exact in
    fp16, rows above zero: what a weight's rounding loses adds up.  The residual takes away the result
    rounded to its type, so that what is left shows sums off by 2^-15.

    Products are exact in fp32; sums of k of them are off by k 2^-24 of the sum (k + 8 with joins), every
    change of scale by a quotient (2^-23 + 2^-24) and a product (2^-24) more: 2^-22 a group."""
    k = -(-k // g) * g
    ng = k // g
    ge = gen(m + n + k + g)
    code = torch.randint(1, 16, (n, ng), generator=ge)
    words = sum(code.repeat_interleave(g // 8, 1) << (4 * i) for i in range(8))
    qw = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()
    sc = scattered_scales(ge, n, ng)
    qz = torch.zeros(n, -(-ng // 8), dtype=torch.int32)
    x = (1 + torch.rand(m, k, generator=ge)).to(dt)
    v = x.double().view(m, ng, g).sum(2) @ (code.double() * sc.double()).t()
    res = (-v).to(dt)
    fn = P.awq_linear_w4a16_act_bf16 if dt is BF16 else P.awq_linear_w4a16_act
    y = fn(x.to(DEV), qw.to(DEV), sc.to(DEV), qz.to(DEV), residual=res.to(DEV), g=g)
    left = v + res.double()
    R.check(y, left, ((k + 8) * 2.0 ** -24 + ng * 2.0 ** -22) * v + R.HALF[dt] * 1.01 * left.abs() + 2.0 ** -25, (m, n, k, g, dt))
    assert bool((y[:, 3] == 0).all())


@pytest.mark.parametrize("g", [128, 64, 32])
@pytest.mark.parametrize("m", [3, 5, 12, 40, 140, 600])
@pytest.mark.parametrize("inv", [False, True])
def test_rows_with_infinities(P, m, g, inv):
    """As in float64: infinite with the weight's sign, NaN where the weight is zero; other rows as ever."""
    n, k = 200, 384
    ge = gen(m + g)
    qw, sc, qz = R.packed(ge, (), n, k, g)
    sc[5] = 0
    sc[:9, (k - 40) // g] = 0                                           # the group of the last row's infinity
    w = R.weights(qw, sc, qz, g)
    x = torch.randn(m, k, generator=ge).half()
    x[1, 7], x[m - 1, k - 40], x[0, 130] = torch.inf, -torch.inf, torch.nan
    iv = torch.full((k,), 0.5).half() if inv else None
    for act in ("none", "silu", "gelu"):
        y = P.awq_linear_w4a16_act(x.to(DEV), qw.to(DEV), sc.to(DEV), qz.to(DEV), None if iv is None else iv.to(DEV),
                                   act=act, g=g).cpu()
        v, bound = R.linear(x, w, iv, None, act, False, None, F16)
        odd = [0, 1, m - 1]
        for i in odd:
            assert torch.equal(y[i].isnan(), v[i].isnan()) and torch.equal(y[i] == torch.inf, v[i] == torch.inf), (i, act)
            assert torch.equal(y[i] == -torch.inf, v[i] == -torch.inf), (i, act)
        rest = [i for i in range(m) if i not in odd]
        assert len(rest) == m - 3
        R.check(y[rest], v[rest], bound[rest], (m, g, act))


@pytest.mark.parametrize("down", [0, 3, 8, 10])
@pytest.mark.parametrize("rows", [1, 4])
@pytest.mark.parametrize("k,g", [(1024, 128), (320, 64), (192, 32)])
def test_small_products_with_the_inverse_scale(P, rows, k, g, down):
    """Rows times 2^-down: what fp16 loses of x inv_s16, 2^-20 of it, is below fp16's last place from 2^-4 on.

    Even channels give (1 + 2^-10)^2, odd ones -(1 + 2^-9), times a power of two: equal once rounded, 2^-20 of
    it apart; every sum is exact in fp32, and so is the result times scales of 2^down."""
    n = 33
    x, inv = torch.full((rows, k), 1 + 2.0 ** -9), torch.ones(k)
    x[:, ::2], inv[::2] = 1 + 2.0 ** -10, 1 + 2.0 ** -10
    x *= 2.0 ** (torch.arange(rows) - down)[:, None]
    words = [sum(8 << (4 * j) for j in range(min(8, k // g - 8 * i))) for i in range(-(-k // (8 * g)))]
    qz = torch.tensor([w - 2 ** 32 if w >= 2 ** 31 else w for w in words]).int().repeat(n, 1)
    qw = torch.full((n, k // 8), 0x79797979, dtype=torch.int32)                      # q - z = 1, -1, 1 ..
    sc = torch.full((n, k // g), 2.0 ** down).half()
    y = P.awq_linear_w4a16_act(*(t.to(DEV) for t in (x.half(), qw, sc, qz, inv.half())), g=g)
    want = (k * 2.0 ** -21 * 2.0 ** torch.arange(rows, dtype=torch.float64))[:, None].expand(rows, n)
    assert torch.equal(y.cpu().double(), want)


def wide_packed(lead, n, k, seed):
    """Packed weights of many rows, made on the device (g = 64)."""
    ge = torch.Generator(device=DEV).manual_seed(seed)
    bits = lambda *shape: torch.randint(-2 ** 31, 2 ** 31 - 1, shape, generator=ge, dtype=torch.int32, device=DEV)
    sc = torch.rand(*lead, n, k // 64, generator=ge, dtype=F16, device=DEV) * 0.1
    ng = k // 64
    qz = bits(*lead, n, -(-ng // 8))
    if ng % 8:
        qz[..., -1] &= (1 << (4 * (ng % 8))) - 1
    return bits(*lead, n, k // 8), sc, qz


def test_few_rows_of_more_columns_than_streaming_launches(P):
    """1024 experts of 131072 outputs and a row each; one matrix of 2^27 - 1 outputs, packed just below 4 GiB."""
    k = 64
    ge = gen(9)
    for e, n in ((1024, 131072), (1, (1 << 27) - 1)):
        rows = 1024 if e > 1 else 2
        p = wide_packed((e,), n, k, e)
        x = torch.randn(rows, k, generator=ge).half()
        if e > 1:
            y = P.awq_moe_linear_w4a16(x.to(DEV), *p, torch.arange(e + 1, dtype=torch.int32, device=DEV), g=k)
        else:
            y = P.awq_linear_w4a16_act(x.to(DEV), *(t[0] for t in p), g=k)
        cols = torch.cat((torch.arange(100), torch.randint(0, n, (300,), generator=ge), torch.arange(n - 100, n)))
        for r in (0, 1, rows // 2, rows - 1):
            j = r if e > 1 else 0
            w = R.weights(*(t[j][cols.to(DEV)].cpu() for t in p), k)
            v, bound = R.linear(x[r:r + 1], w, None, None, "none", False, None, F16)
            R.check(y[r:r + 1][:, cols.to(DEV)], v, bound, (e, r))
        del p, y


@pytest.mark.parametrize("counts", [[0] * 20 + [70, 1, 0, 37] + [2] * 16, [33] + [0] * 9, [3] * 40 + [130] + [0] * 30,
                                    [1, 64, 0, 0, 65] + [0] * 40], ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("gather", [False, True])
def test_streaming_of_experts_with_many_rows(P, counts, gather):
    """Up to six rows to an expert on average, and more than four tiles of eight rows at some."""
    assert sum(counts) + 3 <= 6 * len(counts)
    grouped(P, counts, 200, 256, 128, F16, gather, "silu", True, True, False)
    grouped(P, counts, 333, 192, 64, BF16, gather, "none", False, True, True)
    grouped(P, counts, 264, 96 * 2, 32, F16, gather, "gelu", False, False, True, topk=3)


@pytest.mark.parametrize("dt,inv", [(F16, False), (BF16, False), (F16, True)])
@pytest.mark.parametrize("e,rows,n,k", [(2, (1 << 25) + 100, 8, 64), (1024, 6144, 2, 350080)])
def test_rows_of_x_beyond_31_bits(P, e, rows, n, k, dt, inv):
    """x of more than 2^31 elements, row by row: tiles (as it is and converted) and streaming."""
    assert rows * k > 1 << 31
    p = wide_packed((e,), n, k, rows)
    ge = torch.Generator(device=DEV).manual_seed(k)
    x = torch.empty(rows, k, dtype=dt, device=DEV)
    for part in x.split(rows // 8):
        part.copy_(torch.randn(part.shape, generator=ge, device=DEV).clamp_(-8, 8))
    iv = torch.full((k,), 0.5, dtype=F16, device=DEV) if inv else None
    offsets = torch.tensor([rows * j // e for j in range(e + 1)], dtype=torch.int32, device=DEV)
    fn = P.awq_moe_linear_w4a16_bf16 if dt is BF16 else P.awq_moe_linear_w4a16
    y = fn(x, *p, offsets, inv_s16=iv, g=64)
    for j in (0, e - 1):
        w = R.weights(*(t[j].cpu() for t in p), 64)
        a, z = int(offsets[j]), int(offsets[j + 1])
        at = torch.unique(torch.tensor([a, a + 1, max(a, z - 1000), z - 2, z - 1] + [r for r in ((1 << 31) // k, (1 << 31) // k + 1) if a <= r < z]))
        # bf16 values below fp16's normal range lose up to 2^-25 each
        v, bound = R.linear(x[at.to(DEV)].cpu(), w, None if iv is None else iv.cpu(), None, "none", False, None, dt)
        R.check(y[at.to(DEV)], v, bound, (e, rows, dt, inv, j))


@pytest.mark.parametrize("g", [128, 64, 32])
@pytest.mark.parametrize("m,n,k", [(2, 48, 640), (12, 40, 640), (40, 40, 640), (300, 520, 640), (2000, 4096, 640), (2000, 4096, 768)])
def test_scales_at_their_ends(P, m, n, k, g):
    """Groups of 2^-24, of subnormal and of large scales next to each other, one of NaN: sums of rows of each
    alone and of all, every change of scale up to 2^36."""
    ge = gen(m + n + k + g)
    ng = k // g
    qw, _, qz = R.packed(ge, (), n, k, g)
    ends = torch.tensor([2.0 ** -24, 5 * 2.0 ** -24, 2.0 ** -14, 0.01, 1.0, 900.0, 4095.0])
    sc = ends[torch.randint(0, len(ends), (n, ng), generator=ge)].half()
    for i, v in enumerate(ends):
        sc[i] = v                                                       # rows of one scale alone
    sc[8, ng // 2], sc[9, 0], sc[10, ng - 1] = torch.nan, torch.nan, torch.nan
    x = (torch.randn(m, k, generator=ge) / 8).to(BF16)
    x = torch.where(x.abs() < 2.0 ** -10, torch.full_like(x, 2.0 ** -10), x)
    y = P.awq_linear_w4a16_act_bf16(x.to(DEV), qw.to(DEV), sc.to(DEV), qz.to(DEV), g=g).cpu()
    assert bool(y[:, 8:11].isnan().all())
    keep = [i for i in range(n) if not 8 <= i < 11]
    w = R.weights(qw, sc, qz, g)[keep]
    v, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    R.check(y[:, keep], v, ((k + 8) * 2.0 ** -24 + ng * 2.0 ** -22) * mag + R.HALF[BF16] * 1.01 * v.abs() + 1e-37, (m, n, k, g))
