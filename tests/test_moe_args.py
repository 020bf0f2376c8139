"""Argument checks of the linears with an epilogue and of the mixture-of-experts entries (CPU:
every call here is refused, or has nothing to do, before any launch)."""
from __future__ import annotations

import pytest

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from weight_only_int4_awq_amd import _lib
    if not _lib.LIB_PATH.exists():
        from weight_only_int4_awq_amd.build import build
        build()
    return _lib.load()


def status(lib, fn, *a):
    st = getattr(lib, fn)(*a)
    msg = lib.awq_last_error().decode()
    assert (st == 0) == (msg == "")
    if st:
        assert msg.startswith(fn + ":"), msg
    return st


def caller(lib, fn, names, base):
    def call(**kw):
        a = list(base)
        for n, v in kw.items():
            a[names.index(n)] = v
        return status(lib, fn, *a)
    return call


@pytest.mark.parametrize("fn", ["awq_linear_w4a16_act", "awq_linear_w4a16_act_bf16"])
def test_dense_refusals(lib, fn):
    names = ["x", "qw", "sc", "qz", "inv", "bias", "res", "act", "gated", "m", "n", "k", "g", "y", "ws", "wsb", "st"]
    call = caller(lib, fn, names, [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, 0, 1, 4096, 4096, 128, FAKE, None, 0, None])
    for n in ("x", "qw", "sc", "qz", "y"):
        assert call(**{n: None}) == 1
    for kw in (dict(act=-1), dict(act=4), dict(g=16), dict(g=256), dict(k=0), dict(k=96, g=32), dict(k=4160), dict(n=0),
               dict(n=1 << 31), dict(m=-1), dict(m=(1 << 27) + 1), dict(n=1 << 21), dict(n=1 << 20, gated=1),
               dict(m=1 << 26, n=4096)):
        assert call(**kw) == 2, kw
    for kw in (dict(x=FAKE + 8), dict(qw=FAKE + 4), dict(inv=FAKE + 2), dict(sc=FAKE + 2), dict(qz=FAKE + 1),
               dict(bias=FAKE + 1), dict(res=FAKE + 1), dict(y=FAKE + 1)):
        assert call(**kw) == 3, kw
    assert call(m=0, x=None, y=None) == 0
    need = lib.awq_linear_act_workspace_size(2048, 4096, 4096, 128, 0, 1, 0)
    assert need > 0
    big = dict(m=2048)
    assert call(**big) == 4 and call(ws=FAKE, wsb=need - 1, **big) == 4 and call(ws=FAKE + 128, wsb=1 << 40, **big) == 3


@pytest.mark.parametrize("fn", ["awq_moe_linear_w4a16", "awq_moe_linear_w4a16_bf16"])
def test_grouped_refusals(lib, fn):
    names = ["x", "xr", "qw", "sc", "qz", "inv", "bias", "act", "gated", "e", "off", "slot", "topk", "rows", "n", "k", "g",
             "y", "ws", "wsb", "st"]
    call = caller(lib, fn, names, [FAKE, 4, FAKE, FAKE, FAKE, None, None, 1, 1, 8, FAKE, FAKE, 2, 8, 1024, 4096, 128, FAKE,
                                   None, 0, None])
    for n in ("x", "qw", "sc", "qz", "y", "off"):
        assert call(**{n: None}) == 1
    for kw in (dict(e=0), dict(e=1025), dict(topk=0), dict(topk=33), dict(rows=-1), dict(rows=(1 << 27) + 1), dict(xr=0),
               dict(xr=-1), dict(xr=1 << 20), dict(g=8), dict(k=100), dict(n=0), dict(act=9), dict(n=1 << 20)):
        assert call(**kw) == 2, kw
    for kw in (dict(x=FAKE + 2), dict(qw=FAKE + 8), dict(off=FAKE + 2), dict(slot=FAKE + 1), dict(bias=FAKE + 1)):
        assert call(**kw) == 3, kw
    assert call(rows=0, off=None, x=None) == 0
    need = lib.awq_moe_linear_workspace_size(4096, 4096, 8, 1024, 4096, 128, 1, 1, 0)
    assert need >= 4096 * 4096 * 2
    many = dict(rows=4096, slot=None, inv=FAKE)
    assert call(**many) == 4 and call(ws=FAKE, wsb=need - 1, **many) == 4 and call(ws=FAKE + 16, wsb=1 << 40, **many) == 3


def test_route_refusals(lib):
    names = ["x", "type", "t", "e", "topk", "sc", "rn", "scale", "ids", "w", "off", "rs", "sr", "ws", "wsb", "st"]
    call = caller(lib, "awq_moe_route", names, [FAKE, 0, 8, 8, 2, 0, 1, 1.0, FAKE, FAKE, FAKE, FAKE, FAKE, None, 0, None])
    for n in ("x", "ids", "w", "off", "rs", "sr"):
        assert call(**{n: None}) == 1
    for kw in (dict(type=-1), dict(type=3), dict(sc=2), dict(e=0), dict(e=1025), dict(topk=0), dict(topk=9),
               dict(topk=33, e=64), dict(t=-1), dict(t=(1 << 24) + 1), dict(t=1 << 24, topk=32, e=64), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**kw) == 2, kw
    for kw in (dict(x=FAKE + 2), dict(type=1, x=FAKE + 1), dict(ids=FAKE + 2), dict(w=FAKE + 1), dict(off=FAKE + 3),
               dict(rs=FAKE + 2), dict(sr=FAKE + 2)):
        assert call(**kw) == 3, kw
    need = lib.awq_moe_route_workspace_size(5000, 8)
    assert need > 0 and lib.awq_moe_route_workspace_size(1, 8) == 0
    assert call(t=5000) == 4 and call(t=5000, ws=FAKE, wsb=need - 1) == 4 and call(t=5000, ws=FAKE + 8, wsb=need) == 3
    for bad in ((-1, 8), ((1 << 24) + 1, 8), (5000, 0), (5000, 1025)):
        assert lib.awq_moe_route_workspace_size(*bad) == 0


@pytest.mark.parametrize("fn", ["awq_moe_combine", "awq_moe_combine_bf16"])
def test_combine_refusals(lib, fn):
    names = ["rows", "r", "w", "sr", "res", "t", "n", "topk", "y", "st"]
    call = caller(lib, fn, names, [FAKE, 16, FAKE, FAKE, FAKE, 8, 64, 2, FAKE, None])
    for n in ("rows", "w", "sr", "y"):
        assert call(**{n: None}) == 1
    for kw in (dict(topk=0), dict(topk=33), dict(n=0), dict(n=(1 << 24) + 1), dict(t=-1), dict(t=(1 << 24) + 1),
               dict(r=-1), dict(r=(1 << 27) + 1), dict(t=1 << 20, n=4097)):
        assert call(**kw) == 2, kw
    for kw in (dict(rows=FAKE + 1), dict(w=FAKE + 2), dict(sr=FAKE + 2), dict(res=FAKE + 1), dict(y=FAKE + 1)):
        assert call(**kw) == 3, kw
    assert call(t=0, y=None, rows=None) == 0


def test_workspace_sizes(lib):
    f, h = lib.awq_linear_act_workspace_size, lib.awq_moe_linear_workspace_size
    assert f(1, 4096, 4096, 128, 0, 1, 1) == 0
    for bad in ((0, 64, 64, 64, 0, 0, 0), (8, 64, 64, 48, 0, 0, 0), (8, 0, 64, 64, 0, 0, 0), (8, 64, 100, 64, 0, 0, 0),
                (1 << 28, 64, 64, 64, 0, 0, 0)):
        assert f(*bad) == 0, bad
    assert h(16, 8, 8, 1024, 2048, 128, 1, 0, 0) == 0
    for bad in ((0, 8, 8, 64, 64, 64, 0, 0, 0), (8, 0, 8, 64, 64, 64, 0, 0, 0), (8, 8, 0, 64, 64, 64, 0, 0, 0),
                (8, 8, 1025, 64, 64, 64, 0, 0, 0)):
        assert h(*bad) == 0, bad


def test_binding_refuses_host_tensors_and_names():
    torch = pytest.importorskip("torch")
    import weight_only_int4_awq_amd as P
    x = torch.zeros(2, 64, dtype=torch.float16)
    qw, sc, qz = torch.zeros(8, 8, dtype=torch.int32), torch.zeros(8, 1, dtype=torch.float16), torch.zeros(8, 1, dtype=torch.int32)
    off = torch.zeros(2, dtype=torch.int32)
    w, sr = torch.zeros(2, 2), torch.zeros(2, 2, dtype=torch.int32)
    for call in (lambda: P.awq_linear_w4a16_act(x, qw, sc, qz, g=64), lambda: P.awq_moe_route(torch.zeros(4, 8), 2),
                 lambda: P.awq_moe_linear_w4a16(x, qw[None], sc[None], qz[None], off, g=64),
                 lambda: P.awq_moe_combine(x, w, sr)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="act"):
        P.awq_linear_w4a16_act(x, qw, sc, qz, act="relu")
    with pytest.raises(ValueError, match="scoring"):
        P.awq_moe_route(torch.zeros(4, 8), 2, scoring="max")
    for call in (lambda: P.awq_moe_route([[1.0]], 1), lambda: P.awq_linear_w4a16_act([1.0], qw, sc, qz),
                 lambda: P.awq_moe_route(torch.zeros(4, 8, dtype=torch.float64), 2),
                 lambda: P.awq_moe_combine(x, [1.0], sr)):
        with pytest.raises((TypeError, ValueError)):
            call()


def test_binding_refuses_groups_of_nothing():
    torch = pytest.importorskip("torch")
    import weight_only_int4_awq_amd as P
    x = torch.zeros(2, 64, dtype=torch.float16)
    qw, sc, qz = torch.zeros(8, 8, dtype=torch.int32), torch.zeros(8, 1, dtype=torch.float16), torch.zeros(8, 1, dtype=torch.int32)
    for g in (0, -64):
        with pytest.raises(ValueError, match="g must"):
            P.awq_linear_w4a16_act(x, qw, sc, qz, g=g)
        with pytest.raises(ValueError, match="g must"):
            P.awq_moe_linear_w4a16(x, qw[None], sc[None], qz[None], torch.zeros(2, dtype=torch.int32), g=g)
