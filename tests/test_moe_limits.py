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
