"""CPU oracle for the paged cache held in 8 bits and for the rotary positions: float64 and whole numbers, plain loops.

TEST INFRASTRUCTURE ONLY.  Only the tests and the package smoke check may import it.  The CUDA library never does and
shares no code with it.
"""
from __future__ import annotations

import math

import numpy as np

from oracle import paged_oracle as P

BAD, NON_FINITE = 16, 8
BLOCK, LEAST, MOST = 16, -60, 60
NAN_CODE = 0x7F


def _decode(c: int) -> float:
    sign, exp, man = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
    if exp == 15 and man == 7:
        return math.nan
    return sign * (man * 2.0 ** -9 if exp == 0 else (8 + man) * 2.0 ** (exp - 10))


VALUES = np.array([_decode(c) for c in range(256)])    # of the 256 codes


def to_f64(codes) -> np.ndarray:
    return VALUES[np.asarray(codes, dtype=np.uint8)]


def to_codes(x) -> np.ndarray:
    """Values to the nearest codes, ties to the even one; |x| up to 464 (which rounds to 448), NaN to 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    nan = np.isnan(x)
    a = np.where(nan, 0.0, np.abs(x))
    assert a.size == 0 or a.max() <= 464.0
    mags = VALUES[:0x7F]                               # 0 .. 448, increasing
    hi = np.clip(np.searchsorted(mags, a), 1, 0x7E)
    lo = hi - 1
    up, down = mags[hi] - a, a - mags[lo]
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code |= (np.signbit(x) << 7).astype(np.uint8)
    return np.where(nan, np.uint8(NAN_CODE), code)


def exponent(amax: float) -> int:
    """The least e of LEAST .. MOST with amax <= 448 * 2^e."""
    e = LEAST
    while e < MOST and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def scale_ok(s: float) -> bool:
    """A power of two from 2^LEAST to 2^MOST."""
    return math.isfinite(s) and 2.0 ** LEAST <= s <= 2.0 ** MOST and math.frexp(s)[0] == 0.5


def values(cache, scale, page_size) -> np.ndarray:
    """codes [P, H, S, D] and scales [P, H, S / 16] as float64 values."""
    s = np.asarray(scale, dtype=np.float64)
    return to_f64(cache) * np.repeat(s, BLOCK, axis=2)[..., None]


def append(k, v, table, q_start, kv_len, caches, scales, dtype):
    """k, v [T, H, D] patterns; caches and scales pairs of arrays.  Returns new pairs and the flags."""
    flags = 0
    out_c, out_s = [c.copy() for c in caches], [s.copy() for s in scales]
    P_, H, S, _ = caches[0].shape
    for b in range(len(kv_len)):
        r0, n, L = int(q_start[b]), int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        p0 = L - n
        for j0 in range(max(p0, 0) // BLOCK * BLOCK, L if n > 0 else 0, BLOCK):
            first, last = max(p0, j0, 0), min(L, j0 + BLOCK)
            page, off = int(table[b][j0 // S]), j0 % S
            if not 0 <= page < P_:
                flags |= BAD
                continue
            for which, rows in enumerate((k, v)):
                for h in range(H):
                    x = P.to_f64(rows[r0 + first - p0:r0 + last - p0, h], dtype)
                    good = np.abs(x) <= 448.0 * 2.0 ** MOST
                    if not good.all():
                        flags |= NON_FINITE
                    was = float(out_s[which][page, h, off // BLOCK])
                    s = 2.0 ** exponent(np.abs(x[good]).max(initial=0.0))
                    held = out_c[which][page, h, off:off + first - j0]
                    if first > j0:
                        if not scale_ok(was):
                            flags, was = flags | BAD, 2.0 ** LEAST
                        s = max(s, was)
                        if s != was:
                            out_c[which][page, h, off:off + first - j0] = to_codes(to_f64(held) * (was / s))
                    out_c[which][page, h, off + first - j0:off + last - j0] = to_codes(np.where(good, x / s, np.nan))
                    out_s[which][page, h, off // BLOCK] = s
    return out_c, out_s, flags


def gather(vals, table_row, L, g):
    """Positions 0 .. L - 1 of head g: zeros where the page is out of range."""
    S = vals.shape[2]
    pages = np.asarray(table_row[:max(1, -(-L // S))], dtype=np.int64)
    sane = (pages >= 0) & (pages < vals.shape[0])
    x = vals[np.where(sane, pages, 0), g]
    return np.where(sane[:, None, None], x, 0.0).reshape(-1, vals.shape[3])[:L]


def attention(q, k_vals, v_vals, table, q_start, kv_len, window=0, sinks=0, dtype="bf16"):
    """q [T, Hq, D] patterns over value caches [P, H, S, D]; returns o, mag and smax as paged_oracle.attention does."""
    T, Hq, D = q.shape
    H = k_vals.shape[1]
    G = Hq // H
    o, mag, smax = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan), np.zeros((T, Hq))
    for b in range(len(kv_len)):
        r0, r1, L = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        if r0 == r1:
            continue
        p = L - r1 + np.arange(r0, r1)[:, None]
        j = np.arange(L)[None, :]
        see = j <= p
        if window > 0:
            see &= (j > p - window) | (j < sinks)
        some = see.any(1)
        for g in range(H):
            kk, vv = gather(k_vals, table[b], L, g), gather(v_vals, table[b], L, g)
            seen = see.any(0)
            kk, vv = np.where(seen[:, None], kk, 0.0), np.where(seen[:, None], vv, 0.0)
            for h in range(g * G, (g + 1) * G):
                qq = P.to_f64(q[r0:r1, h], dtype)
                s = np.where(see, qq @ kk.T / math.sqrt(D), -np.inf)
                e = np.exp(s - np.where(some, s.max(1, initial=-np.inf), 0.0)[:, None])
                e /= np.where(some, e.sum(1), 1.0)[:, None]
                bad = ~np.isfinite(vv)
                o[r0:r1, h] = e @ np.where(bad, 0.0, vv)
                mag[r0:r1, h] = e @ np.abs(np.where(bad, 0.0, vv))
                if bad.any():                          # a row has NaN in the dims where a position that it sees has
                    o[r0:r1, h] = np.where((see.astype(float) @ bad) > 0, np.nan, o[r0:r1, h])
                if L > 0:
                    smax[r0:r1, h] = np.where(see, np.abs(qq) @ np.abs(kk).T, 0.0).max(1) / math.sqrt(D)
    return o, mag, smax


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0.0, low=1.0, high=32.0) -> np.ndarray:
    """Radians a position of each pair, in long double."""
    i = np.arange(rot // 2, dtype=np.longdouble)
    base = np.longdouble(base)
    if scaling == "base":
        base = base * np.longdouble(factor) ** (np.longdouble(rot) / (rot - 2))
    w = base ** (-2 * i / rot)
    if scaling == "linear":
        return w / np.longdouble(factor)
    if scaling == "by_parts":
        pi = np.longdouble("3.14159265358979323846264338327950288")
        g = np.clip((np.longdouble(original) * w / (2 * pi) - low) / (np.longdouble(high) - low), 0, 1)
        return g * w + (1 - g) * w / np.longdouble(factor)
    return w


def rotary(x, positions, w, layout, amplitude=1.0):
    """x float64 [T, H, D] turned by positions times w; the angle and its reduction in long double."""
    half = len(w)
    rot = 2 * half
    a, b = (slice(0, half), slice(half, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    angle = np.asarray(positions, dtype=np.longdouble)[:, None] * w[None, :]
    c, s = (np.asarray(f(angle), dtype=np.float64)[:, None, :] * amplitude for f in (np.cos, np.sin))
    y = x.copy()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y
