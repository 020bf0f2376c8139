"""The 8-bit paged KV cache from its definition, in numpy on the CPU (test
infrastructure: imports nothing of the product package).

append() follows the documented arithmetic bit for bit: the rotation is float32 with
every product and sum rounded once, the quotient by the scale is float32 (exact for a
power of two), and then there is the one rounding to an e4m3 code.  attend() is float64 throughout and returns
what the error bound of the kernels needs."""
from __future__ import annotations

import numpy as np


def _decode_table():
    t = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = np.nan if (e == 15 and m == 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        t[c] = -v if s else v
    return t


CODE = _decode_table()
_POS = CODE[:127]                                    # 0 .. 448, ascending


def encode(x):
    """uint8 codes of float64 |x| <= 464 (halfway to the next step above 448), nearest, ties to even."""
    a = np.abs(x)
    i = np.clip(np.searchsorted(_POS, a, side="right") - 1, 0, 125)
    lo, hi = _POS[i], _POS[i + 1]
    mid = (lo + hi) / 2
    up = (a > mid) | ((a == mid) & (i % 2 == 1))
    code = np.where(np.isnan(x), 127, np.where(up, i + 1, i))
    return (code | np.where(np.signbit(x) & ~np.isnan(x), 128, 0)).astype(np.uint8)


def scale_of(amax):
    """2^e, the least e >= -64 with amax <= 448 * 2^e."""
    e = -64
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return np.float32(2.0 ** e)


def rotate(x, cs, rot, inter):
    """x float32 [rows, heads, d], cs float32 [rows, rot]."""
    y = x.copy()
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    ia = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
    ib = ia + 1 if inter else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    with np.errstate(over="ignore", invalid="ignore"):
        y[..., ia] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
        y[..., ib] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return y


def positions(cu, ctx, b):
    return range(cu[b], cu[b + 1]), int(ctx[b]) - (cu[b + 1] - cu[b])


def append(kc, vc, ks, vs, bt, ctx, cu, k, v, table=None, inter=False):
    """Updates kc, vc (uint8) and ks, vs (float32) in place; k, v float32 [rows, hkv, d]."""
    pages, hkv, page, d = kc.shape
    for b in range(len(ctx)):
        rows, first = positions(cu, ctx, b)
        n = len(rows)
        if n == 0:
            continue
        pos = first + np.arange(n)
        kk, vv = k[rows.start:rows.stop].copy(), v[rows.start:rows.stop]
        lost = np.zeros(n, bool)
        if table is not None:
            lost = pos >= table.shape[0]
            cs = table[np.clip(pos, 0, table.shape[0] - 1)]
            kk = rotate(kk, cs, table.shape[1], inter)
        bad = ~(np.isfinite(kk).all(2) & np.isfinite(vv).all(2)) | lost[:, None]      # [n, hkv]
        for j in range(max(0, pos[0]) // page, (pos[-1] // page if pos[-1] >= 0 else -1) + 1):
            if j >= bt.shape[1] or not 0 <= bt[b, j] < pages:
                continue
            at = bt[b, j]
            here = (pos >= 0) & (pos // page == j)
            old = max(0, max(0, first) - j * page)
            for h in range(hkv):
                good = here & ~bad[:, h]
                for x, cache, scale in ((kk, kc[at, h], ks), (vv, vc[at, h].T, vs)):
                    amax = float(np.abs(x[good, h]).max()) if good.any() else 0.0
                    s = scale_of(amax)
                    if old:
                        s = max(s, scale[at, h])
                        if s != scale[at, h]:
                            cache[:old] = encode((CODE[cache[:old]].astype(np.float32) * (scale[at, h] / s)).astype(np.float64))
                    scale[at, h] = s
                    for i in np.nonzero(here)[0]:
                        if bad[i, h]:
                            cache[pos[i] - j * page] = 0x7F if scale is ks else 0
                        else:
                            cache[pos[i] - j * page] = encode((x[i, h] / np.float32(s)).astype(np.float64))


def attend(q, kc, vc, ks, vs, bt, ctx, cu, scale):
    """q float64 [rows, hq, d] -> (out, lse, mag, smag): mag[r, a, c] = sum_t p_t |v_tc|,
    smag[r, a] = the largest scale * sum_c |q_c k_tc| over the visible t.  Rows of no sequence: 0."""
    pages, hkv, page, d = kc.shape
    rows, hq, _ = q.shape
    G = hq // hkv
    out, mag = np.zeros((rows, hq, d)), np.zeros((rows, hq, d))
    lse, smag = np.zeros((rows, hq)), np.zeros((rows, hq))
    for b in range(len(ctx)):
        rr, first = positions(cu, ctx, b)
        if len(rr) == 0:
            continue
        need = -(-int(ctx[b]) // page)
        for h in range(hkv):
            k, v = np.zeros((need * page, d)), np.zeros((need * page, d))
            for j in range(need):
                at = bt[b, j]
                k[j * page:(j + 1) * page] = CODE[kc[at, h]] * float(ks[at, h])
                v[j * page:(j + 1) * page] = (CODE[vc[at, h]] * float(vs[at, h])).T
            for i, r in enumerate(rr):
                m = first + i + 1
                for a in range(h * G, (h + 1) * G):
                    if m <= 0:
                        lse[r, a] = -np.inf
                        continue
                    s = scale * (k[:m] @ q[r, a])
                    top = s.max()
                    e = np.exp(s - top)
                    p = e / e.sum()
                    out[r, a], mag[r, a] = p @ v[:m], p @ np.abs(v[:m])
                    lse[r, a] = top + np.log(e.sum())
                    smag[r, a] = scale * (np.abs(k[:m]) @ np.abs(q[r, a])).max()
    return out, lse, mag, smag


def bounds(out, lse, mag, smag, d, eps):
    """Error bounds of the kernels against attend(), from their arithmetic.

    A score is an fp32 sum of d exact products (d + 1 roundings of at most 2^-24 of
    the sum of magnitudes each), scaled twice and shifted (4 more): |ds| <= (d + 8) 2^-24 smag.
    exp2 of the difference to the running maximum: its argument holds log2 of a
    power-of-two scale exactly and is rounded at a magnitude of at most
    |s| + 64 + |m|, so add 2^-23 (2 smag + 128); the hardware's exp2 and the rescaling
    products add 2^-20 together.  So a weight is off by a factor of 1 +- w with
    w = 2 (ds + ...) (numerator and denominator), and by 2^-11 for its rounding to fp16
    (half a step is 2^-11 of the value); the value product's fp32 sums add 2^-14
    of mag for up to 2^10 additions in a row.  Then the output's own half step eps / 2."""
    ds = (d + 8) * 2.0 ** -24 * smag + 2.0 ** -23 * (2 * smag + 128) + 2.0 ** -20
    to = (2 * ds[..., None] + 2.0 ** -11 + 2.0 ** -14) * mag
    to = to + eps / 2 * (np.abs(out) + to)
    return to, ds + 2.0 ** -22 * (np.abs(np.where(np.isfinite(lse), lse, 0)) + 1) + 2.0 ** -20
