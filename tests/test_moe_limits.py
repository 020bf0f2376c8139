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


def test_grouped_limit_is_that_of_the_tiles(lib):
    """(rows / 32 + min(e, rows)) column blocks of 256 outputs (gated 128), below 2^22, whatever kernel few rows
    to an expert would take.  With inv_s16 a workspace is needed wherever sizes are taken and tiles are used."""
    def need(rows, e, n, gated=0, k=64):
        return lib.awq_moe_linear_workspace_size(rows, rows, e, n, k, 64, gated, 1, 0)
    assert need(1024, 1024, 131072) >= 1024 * 128                          # few rows, wide: tiles
    assert need(6144, 1024, 65536, 1) >= 6144 * 128
    assert need(1024, 1024, 1 << 20) == 0                                  # 1056 * 4096
    assert need(1024, 1024, 3971 * 256) >= 1024 * 128 and need(1024, 1024, 3972 * 256) == 0
    assert need(1024, 1024, 3971 * 128, 1) >= 1024 * 128 and need(1024, 1024, 3972 * 128, 1) == 0
    for fn in ("awq_moe_linear_w4a16", "awq_moe_linear_w4a16_bf16"):
        def call(rows, e, n, gated):
            return getattr(lib, fn)(FAKE, rows, FAKE, FAKE, FAKE, FAKE, None, 0, gated, e, FAKE, None, 1, rows, n, 64, 64,
                                    FAKE, None, 0, None)
        assert call(1024, 1024, 131072, 0) == 4 and call(6144, 1024, 65536, 1) == 4          # no workspace given
        assert call(1024, 1024, 1 << 20, 0) == 2


def test_dense_limits_are_those_of_the_sizes_alone(lib):
    """m n / 4, m k / 8 and the packed weights' 4 GiB: nothing within them is more than a launch holds."""
    def need(m, n, k, gated=0):
        return lib.awq_linear_act_workspace_size(m, n, k, 64, gated, 1, 0)
    def status(m, n, k, gated=0):                                          # without x: 1 where the sizes are taken
        return lib.awq_linear_w4a16_act(None, FAKE, FAKE, FAKE, None, None, None, 0, gated, m, n, k, 64, FAKE, None, 0, None)
    wide = (1 << 27) - 1                                                   # 64 channels: just below 4 GiB
    for m in (1, 8, 9, 16, 17, 64):
        assert status(m, wide, 64) == 1 and status(m, wide // 2, 64, 1) == 1, m
        assert status(m, 1 << 27, 64) == 2 and status(m, 1 << 26, 64, 1) == 2, m
    assert status(1 << 27, 64, 64) == 1 and status((1 << 27) + 1, 64, 64) == 2
    assert status(1 << 27, 65, 64) == 2 and status(1 << 27, 64, 192) == 2  # m n / 4, m k / 8
    assert status(1 << 20, 8192, 64) == 1 and status((1 << 20) + 1, 8192, 64) == 2
    assert status(1 << 20, 8192, 64, 1) == 1 and need(1 << 20, 8192, 64, 1) >= 1 << 27


def test_rows_that_stream(lib):
    """One matrix streams up to 16 rows, and up to 512 where 36 MiB of weights and 2^16 weight rows are read in
    all, 16 rows at a time; with inv_s16 tiles need a workspace and streaming none."""
    def streams(m, n, k, gated=0):
        return lib.awq_linear_act_workspace_size(m, n, k, 128, gated, 1, 0) == 0
    assert streams(16, 14336, 4096, 1) and not streams(17, 14336, 4096, 1)
    assert streams(64, 4096, 4096) and not streams(81, 4096, 4096)         # MiB: 4 passes of 8, 6 of 8
    assert streams(240, 4096, 512) and not streams(241, 4096, 512)         # rows: 15 passes of 4096, 16 of 4096
    assert streams(240, 2048, 512, 1) and not streams(241, 2048, 512, 1)
    assert streams(512, 512, 4096) and not streams(513, 512, 4096)
