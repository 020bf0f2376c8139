"""What the binding asks for of mixture-of-experts calls, and the limits of their sizes (CPU: every call
here is refused before any launch)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("name", ["awq_moe_linear_w4a16", "awq_moe_linear_w4a16_bf16"])
def test_slots_need_their_topk(name):
    """Slots are token * topk + choice: without topk they would be read as tokens."""
    import weight_only_int4_awq_amd as P
    x = torch.zeros(2, 64, dtype=torch.float16)
    packed = (torch.zeros(1, 8, 8, dtype=torch.int32), torch.zeros(1, 8, 1, dtype=torch.float16),
              torch.zeros(1, 8, 1, dtype=torch.int32))
    offsets, slots = torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="topk"):
        getattr(P, name)(x, *packed, offsets, slots, g=64)
    for kw in (dict(row_slot=slots, topk=2), dict(row_slot=slots, topk=1), dict(row_slot=slots[:2]), dict(), dict(topk=1)):
        with pytest.raises(ValueError, match="GPU"):                        # past it: tensors of the host
            getattr(P, name)(x, *packed, offsets, g=64, **kw)


FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from weight_only_int4_awq_amd import _lib
    if not _lib.LIB_PATH.exists():
        from weight_only_int4_awq_amd.build import build
        build()
    return _lib.load()


@pytest.mark.parametrize("fn", ["awq_moe_combine", "awq_moe_combine_bf16"])
def test_combine_limit_goes_by_the_threads_of_a_token(lib, fn):
    """n / 8 where all rows are of aligned 16 bytes, else n: 2^31 in all.  Within it the missing weights are named."""
    def call(t, n, rows=FAKE, residual=FAKE, y=FAKE):
        return getattr(lib, fn)(rows, 16, None, FAKE, residual, t, n, 2, y, None)
    assert call(1 << 20, 4096) == 1 and call(1 << 22, 4096) == 1 and call((1 << 22) + 1, 4096) == 2
    assert call(1 << 20, 4096, residual=None) == 1
    for off in (dict(rows=FAKE + 2), dict(residual=FAKE + 8), dict(y=FAKE + 2)):
        assert call(1 << 19, 4096, **off) == 1 and call((1 << 19) + 1, 4096, **off) == 2, off
    assert call(1 << 20, 2047) == 1 and call(1 << 20, 2049) == 2
