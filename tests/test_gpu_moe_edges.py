"""Edges of the linears with an epilogue, of products grouped by expert and of their combination,
against float64 (tests/moe_ref.py) or to the bit."""
from __future__ import annotations

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
