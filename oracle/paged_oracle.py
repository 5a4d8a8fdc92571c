"""CPU oracle for the paged key/value cache: the tables of a step, the append, and the attention.

TEST INFRASTRUCTURE ONLY.  Plain loops over sequences and float64 arithmetic; only the tests and the
package smoke check may import it.  The CUDA library never does and shares no code with it.
"""
from __future__ import annotations

import math

import numpy as np

BAD = 16   # a length, page or slot out of range


def to_f64(bits, dtype: str) -> np.ndarray:
    """16-bit patterns (uint16) -> exact float64 values."""
    b = np.ascontiguousarray(bits).astype(np.uint16)
    if dtype == "fp16":
        return b.view(np.float16).astype(np.float64)
    return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def plan(ctx_len, new_len, free_pages, n_free, table, page_size, num_pages, T, positions, slots):
    """Tables of one step (include/gqa_paged.h).  table [B, M], positions and slots [T] give the entries
    that the call leaves as they were.  Returns a dict with the outputs and the error bits."""
    table, positions, slots = table.copy(), positions.copy(), slots.copy()
    B, M = table.shape
    cap = M * page_size
    flags = 0
    if not 0 <= n_free <= len(free_pages):
        flags, n_free = BAD, min(max(n_free, 0), len(free_pages))
    q_start, kv_len, row, taken = [], [], 0, 0
    for b in range(B):
        c, n = int(ctx_len[b]), int(new_len[b])
        if c < 0 or n < 0 or max(c, 0) + max(n, 0) > cap:
            flags = BAD
        c, n = min(max(c, 0), cap), max(n, 0)
        kv = min(c + n, cap)
        q_start.append(min(row, T))
        kv_len.append(kv)
        for i in range(-(-c // page_size), -(-kv // page_size)):
            page = int(free_pages[n_free - 1 - taken]) if taken < n_free else -1
            taken += 1
            if not 0 <= page < num_pages:
                flags, page = BAD, -1
            table[b, i] = page
        for i in range(n):
            if row + i >= T:
                flags = BAD
                break
            p = c + i
            positions[row + i] = p
            page = int(table[b, p // page_size]) if p < kv else -1
            if not 0 <= page < num_pages:
                flags, page = BAD, -1
            slots[row + i] = page * page_size + p % page_size if page >= 0 else -1
        row += n
    q_start.append(min(row, T))
    return {"table": table, "q_start": np.array(q_start, np.int32), "kv_len": np.array(kv_len, np.int32),
            "positions": positions, "slots": slots, "n_free": max(0, n_free - taken), "flags": flags}


def append(k, v, slots, rows, k_cache, v_cache):
    """k, v [T, H, D] patterns into copies of the caches [P, H, S, D]; rows at or past `rows` and slots of
    -1 are skipped."""
    k_cache, v_cache = k_cache.copy(), v_cache.copy()
    P, _, S, _ = k_cache.shape
    flags = 0
    for t in range(rows):
        s = int(slots[t])
        if not 0 <= s < P * S:
            flags |= 0 if s == -1 else BAD
            continue
        k_cache[s // S, :, s % S] = k[t]
        v_cache[s // S, :, s % S] = v[t]
    return k_cache, v_cache, flags


def visible(p: int, L: int, window: int, sinks: int) -> np.ndarray:
    """Positions that the token at position p sees, of the L cached ones."""
    j = np.arange(L)
    see = j <= p
    if window > 0:
        see &= (j > p - window) | (j < sinks)
    return j[see]


def attention(q, k_cache, v_cache, table, q_start, kv_len, window=0, sinks=0, dtype="bf16"):
    """q [T, Hq, D], caches [P, H, S, D] (patterns); returns o float64 [T, Hq, D] (NaN in the rows of no
    sequence), mag (the same attention over |V|) and smax [T, Hq] (the largest sum_i |q_i k_i| / sqrt(D)
    over a row's visible positions, which bounds the rounding of its scores)."""
    T, Hq, D = q.shape
    P, H, S, _ = k_cache.shape
    G = Hq // H
    o, mag, smax = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan), np.zeros((T, Hq))
    for b in range(len(kv_len)):
        r0, r1, L = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        if r0 == r1:
            continue
        pages = np.asarray(table[b][:max(1, -(-L // S))], dtype=np.int64)
        sane = (pages >= 0) & (pages < P)
        rows = np.where(sane, pages, 0)
        for g in range(H):
            kk = to_f64(np.where(sane[:, None, None], k_cache[rows, g], 0), dtype).reshape(-1, D)[:L]
            vv = to_f64(np.where(sane[:, None, None], v_cache[rows, g], 0), dtype).reshape(-1, D)[:L]
            for t in range(r0, r1):
                see = visible(L - (r1 - t), L, window, sinks)
                for h in range(g * G, (g + 1) * G):
                    if len(see) == 0:
                        o[t, h] = mag[t, h] = 0.0
                        continue
                    qq = to_f64(q[t, h], dtype)
                    s = kk[see] @ qq / math.sqrt(D)
                    e = np.exp(s - s.max())
                    e /= e.sum()
                    o[t, h] = e @ vv[see]
                    mag[t, h] = e @ np.abs(vv[see])
                    smax[t, h] = (np.abs(kk[see]) @ np.abs(qq)).max() / math.sqrt(D)
    return o, mag, smax
