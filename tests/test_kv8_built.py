"""What the library holds for the 8-bit KV cache: the kernels that a call can reach, error texts (CPU)."""
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


def test_error_texts_belong_to_their_thread():
    """Refused calls of two threads, one text each, read back after both have failed."""
    import ctypes as C
    import threading

    from weight_only_int4_awq_amd import _lib
    if not _lib.LIB_PATH.exists():
        from weight_only_int4_awq_amd.build import build
        build()
    lib = _lib.load()
    both, texts = threading.Barrier(2), [None, None]

    def refuse(i):
        c = _lib.Kv8Cache(page=(16, 64)[i], hkv=8, d=(128, 96)[i], pages=1)
        st = lib.awq_attn_kv8(C.byref(c), 1, 1, None, 0, 8, 1.0, None, 0, None, None, 0, None)
        both.wait(30)
        texts[i] = st, lib.awq_last_error().decode()

    threads = [threading.Thread(target=refuse, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert texts[0][0] == texts[1][0] == 2 and "page=16" in texts[0][1] and "d=96" in texts[1][1]
