"""The attention kernels that the library holds are those that a call can reach (CPU)."""
from __future__ import annotations

import re


def test_line_kernels_are_those_of_the_plan():
    """Tiles of 16 columns: eight or two waves, the cache read once (one tile per sequence) or not.
    Tiles of 32 stand for more than 64 columns, so a sequence has several: eight waves, never once."""
    from weight_only_int4_awq_amd import _lib
    if not _lib.LIB_PATH.exists():
        from weight_only_int4_awq_amd.build import build
        build()
    built = {tuple(int(x) for x in m) for m in
             re.findall(rb"attn_kv8_line_kernelILi(\d+)ELb([01])ELi(\d+)ELi(\d+)ELb([01])E", _lib.LIB_PATH.read_bytes())}
    forms = [(16, 8, 1), (16, 8, 0), (16, 2, 1), (16, 2, 0), (32, 8, 0)]
    assert built == {(d, bf, *f) for d in (64, 128) for bf in (0, 1) for f in forms}
