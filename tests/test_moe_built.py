"""What the library holds for linears with an epilogue: the kernels that a call can reach (CPU)."""
from __future__ import annotations

import re


def test_kernels_are_those_of_the_plan():
    """Streaming: tiles of 8 or 16 rows, scales by quads only where a group is a block (g = 128).
    Tiles: 32, 64 or 128 rows by K-steps of 64, one or two K groups; 32 rows by 128 where half a
    K-step is of one group (g >= 64)."""
    from weight_only_int4_awq_amd import _lib
    if not _lib.LIB_PATH.exists():
        from weight_only_int4_awq_amd.build import build
        build()
    data = _lib.LIB_PATH.read_bytes()
    stream = {tuple(int(x) for x in m) for m in re.findall(rb"linear_act_stream_kernelILi(\d+)ELi(\d+)ELb([01])E", data)}
    assert stream == {(g, tm, q) for g in (32, 64, 128) for tm in (8, 16) for q in (0, 1) if not q or g == 128}
    tile = {tuple(int(x) for x in m) for m in re.findall(rb"linear_act_tile_kernelILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)E", data)}
    assert tile == {(g, kg, bm, bk) for g in (32, 64, 128) for kg in (1, 2) for bm in (32, 64, 128) for bk in (64, 128)
                    if bk == 64 or (bm == 32 and g >= 64)}


def test_routing_kernels_are_those_of_the_plan():
    """Lanes of 8, 16 or 32 experts where four tokens share a wave; else 1 to 16 experts to a lane."""
    from weight_only_int4_awq_amd import _lib
    if not _lib.LIB_PATH.exists():
        from weight_only_int4_awq_amd.build import build
        build()
    data = _lib.LIB_PATH.read_bytes()
    for name, held in ((b"moe_route_rows_kernel", {8, 16, 32}), (b"moe_route_kernel", {1, 2, 4, 8, 16}),
                       (b"moe_route_small_kernel", {1, 2, 4, 8, 16})):
        assert {int(x) for x in re.findall(name + rb"ILi(\d+)E", data)} == held, name
