"""Argument checks of the 8-bit KV cache's entries (CPU: every call here is refused before
any launch), and the reference of its GPU tests pinned against torch's e4m3 conversion."""
from __future__ import annotations

import ctypes as C

import numpy as np
import pytest

from tests import kv8_ref as R

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from weight_only_int4_awq_amd import _lib
    if not _lib.LIB_PATH.exists():
        from weight_only_int4_awq_amd.build import build
        build()
    return _lib.load()


def cache(**kw):
    from weight_only_int4_awq_amd import _lib
    f = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, block_table=FAKE, cu_q=FAKE, ctx=FAKE, pages=10,
             max_pages=4, b=2, page=64, hkv=8, d=128)
    f.update(kw)
    return _lib.Kv8Cache(**f)


BAD_CACHES = [(dict(page=16), 2), (dict(page=96), 2), (dict(page=512), 2), (dict(d=96), 2), (dict(d=256), 2),
              (dict(hkv=0), 2), (dict(hkv=1025), 2), (dict(pages=0), 2), (dict(pages=1 << 31), 2),
              (dict(max_pages=-1), 2), (dict(max_pages=1 << 26), 2), (dict(b=-1), 2), (dict(b=65537), 2),
              (dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1), (dict(v_scale=None), 1),
              (dict(block_table=None), 1), (dict(ctx=None), 1), (dict(k=FAKE + 8), 3), (dict(v=FAKE + 1), 3),
              (dict(k_scale=FAKE + 2), 3), (dict(cu_q=FAKE + 1), 3), (dict(ctx=FAKE + 3), 3),
              (dict(block_table=FAKE + 2), 3)]


def status(lib, fn, *a):
    st = getattr(lib, fn)(*a)
    msg = lib.awq_last_error().decode()
    assert (st == 0) == (msg == "")
    if st:
        assert msg.startswith(fn + ":"), msg
    return st


@pytest.mark.parametrize("fn", ["awq_kv8_append", "awq_kv8_append_bf16"])
def test_append_refusals(lib, fn):
    names = ["rows", "q", "qs", "hq", "k", "ks", "v", "vs", "rope", "pos", "rot", "il", "o", "os", "st"]
    base = [5, FAKE, 4096, 32, FAKE, 1024, FAKE, 1024, FAKE, 100, 128, 0, FAKE, 4096, None]

    def call(c=None, **kw):
        a = list(base)
        for n, x in kw.items():
            a[names.index(n)] = x
        return status(lib, fn, C.byref(c if c is not None else cache()), *a)

    assert status(lib, fn, None, *base) == 1
    for kw, st in BAD_CACHES:
        assert call(cache(**kw)) == st, kw
    assert call(rows=-1) == 2 and call(rows=(1 << 24) + 1) == 2
    assert call(k=None) == 1 and call(v=None) == 1 and call(o=None) == 1
    assert call(ks=1016) == 2 and call(vs=512) == 2 and call(qs=4088) == 2 and call(os=8) == 2
    assert call(ks=1028) == 3 and call(k=FAKE + 8) == 3 and call(v=FAKE + 2) == 3 and call(q=FAKE + 4) == 3
    assert call(hq=0) == 2 and call(hq=12) == 2
    assert call(rot=8) == 2 and call(rot=144) == 2 and call(rot=72) == 2
    assert call(pos=0) == 2 and call(rope=FAKE + 4) == 3
    # nothing to do is no error, and nothing is launched
    assert call(rows=0, k=None, v=None, q=None, o=None) == 0
    assert call(cache(b=0, ctx=None, block_table=None)) == 0


@pytest.mark.parametrize("fn", ["awq_attn_kv8", "awq_attn_kv8_bf16"])
def test_attention_refusals(lib, fn):
    names = ["rows", "mq", "q", "qs", "hq", "scale", "o", "os", "lse", "ws", "wsb", "st"]
    base = [5, 1, FAKE, 4096, 32, 0.1, FAKE, 4096, None, None, 0, None]

    def call(c=None, **kw):
        a = list(base)
        for n, x in kw.items():
            a[names.index(n)] = x
        return status(lib, fn, C.byref(c if c is not None else cache()), *a)

    assert status(lib, fn, None, *base) == 1
    for kw, st in BAD_CACHES:
        assert call(cache(**kw)) == st, kw
    assert call(rows=-1) == 2 and call(mq=0) == 2 and call(hq=9) == 2 and call(hq=-8) == 2
    assert call(rows=1 << 24, hq=128) == 2
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == 2
    assert call(q=None) == 1 and call(o=None) == 1
    assert call(qs=4088) == 2 and call(os=4000) == 2 and call(qs=4100) == 3 and call(q=FAKE + 2) == 3
    assert call(o=FAKE + 8) == 3 and call(lse=FAKE + 2) == 3
    assert call(rows=0, q=None, o=None) == 0
    # a long context may be split: partial results need the workspace
    long = cache(max_pages=1000)
    need = lib.awq_attn_kv8_workspace_size(2, 5, 32, 8, 128, 64, 1000, 1)
    assert need > 0
    assert call(long) == 4 and call(long, ws=FAKE, wsb=need - 1) == 4 and call(long, ws=FAKE + 128, wsb=need) == 3


def test_workspace_sizes(lib):
    f = lib.awq_attn_kv8_workspace_size
    assert f(1, 1, 32, 8, 128, 64, 4, 1) == 0                       # too short to be split
    assert f(1, 1, 32, 8, 128, 64, 2048, 1) > 0
    for bad in ((0, 1, 32, 8, 128, 64, 99, 1), (1, 0, 32, 8, 128, 64, 99, 1), (1, 1, 12, 8, 128, 64, 99, 1),
                (1, 1, 32, 8, 96, 64, 99, 1), (1, 1, 32, 8, 128, 48, 99, 1), (1, 1, 32, 8, 128, 64, -1, 1),
                (1, 1, 32, 8, 128, 64, 99, 0)):
        assert f(*bad) == 0, bad


def test_rope_table_refusals(lib):
    def call(pos=10, rot=64, base=1e4, kind=0, factor=1.0, low=1.0, high=4.0, trained=100.0, t=FAKE):
        return status(lib, "awq_rope_table", pos, rot, base, kind, factor, low, high, trained, t, None)

    assert call(t=None) == 1 and call(t=FAKE + 2) == 3
    assert call(pos=0) == 2 and call(pos=1 << 31) == 2
    for rot in (0, 1, 63, 258):
        assert call(rot=rot) == 2
    for base in (1.0, -5.0, float("nan"), float("inf")):
        assert call(base=base) == 2
    assert call(kind=-1) == 2 and call(kind=4) == 2
    for kind in (1, 2, 3):
        assert call(kind=kind, factor=0.0) == 2 and call(kind=kind, factor=float("inf")) == 2
    for kind in (2, 3):
        assert call(kind=kind, low=0.0) == 2 and call(kind=kind, low=4.0) == 2 and call(kind=kind, trained=-1.0) == 2


def test_binding_refuses_host_tensors_and_shapes():
    torch = pytest.importorskip("torch")
    import weight_only_int4_awq_amd as P
    kc, vc, ks, vs = P.kv8_cache(3, 2, 64, 64, device="cpu")
    assert kc.shape == (3, 2, 64, 64) and vc.dtype == torch.float8_e4m3fn and ks.shape == (3, 2)
    bt, ctx = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q = torch.zeros(1, 4, 64, dtype=torch.float16)
    k = torch.zeros(1, 2, 64, dtype=torch.float16)
    for call in (lambda: P.awq_attn_kv8(q, kc, vc, ks, vs, bt, ctx), lambda: P.awq_kv8_append(k, k, kc, vc, ks, vs, bt, ctx),
                 lambda: P.awq_rope_table(10, 16, device="cpu")):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="scaling"):
        P.awq_rope_table(10, 16, scaling="other")
    with pytest.raises(TypeError):
        P.awq_attn_kv8(q, [1.0], vc, ks, vs, bt, ctx)


def test_reference_codes_are_e4m3():
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, R.CODE, equal_nan=True)
    rng = np.random.default_rng(3)
    x = np.clip(rng.standard_normal(100000) * np.exp(rng.uniform(-9, 5, 100000)), -448, 448).astype(np.float32)
    mids = ((R._POS[1:] + R._POS[:-1]) / 2).astype(np.float32)                  # ties
    for a in (x, mids, -mids):
        want = torch.from_numpy(a).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(R.encode(a.astype(np.float64)), want)
    assert R.scale_of(448.0) == 1.0 and R.scale_of(448.5) == 2.0 and R.scale_of(0.0) == np.float32(2.0 ** -64)


@pytest.mark.parametrize("rows", [1, 40, 5000, 2 ** 31 - 1])
@pytest.mark.parametrize("most", [2 ** 24, 2 ** 40, 2 ** 59 + 1, 2 ** 63 - 1])
def test_workspace_size_for_any_most_rows(lib, rows, most):
    """max_q times the heads of a key/value head need not fit in 64 bits."""
    f = lib.awq_attn_kv8_workspace_size
    size = f(3, rows, 32, 8, 128, 64, 2048, most)
    assert size == f(3, rows, 32, 8, 128, 64, 2048, 2 ** 20)
    assert (size > 0) == (rows <= 2 ** 24)                          # beyond the limit of rows there is none


@pytest.mark.parametrize("fn", ["awq_kv8_append", "awq_kv8_append_bf16", "awq_attn_kv8", "awq_attn_kv8_bf16"])
@pytest.mark.parametrize("b,rows,hkv", [(65536, 5, 64), (2049, 2049, 1024), (2, 1 << 24, 16), (2, (1 << 17) + 1, 1024)])
def test_more_than_one_launch_holds_is_refused(lib, fn, b, rows, hkv):
    c = cache(b=b, hkv=hkv)
    if "append" in fn:
        args = [rows, None, 0, hkv, FAKE, hkv * 128, FAKE, hkv * 128, None, 0, 0, 0, None, 0, None]
    else:
        args = [rows, rows, FAKE, hkv * 128, hkv, 1.0, FAKE, hkv * 128, None, FAKE, 1 << 40, None]
        assert lib.awq_attn_kv8_workspace_size(b, rows, hkv, hkv, 128, 64, 4000, rows) == 0
    assert status(lib, fn, C.byref(c), *args) == 2
