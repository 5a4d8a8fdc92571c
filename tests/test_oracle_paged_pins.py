"""Pins of the paged-cache oracle: closed forms, hand-built tables and the contiguous attention oracle."""
import numpy as np
import pytest

import synth
from oracle import attention_oracle as A
from oracle import paged_oracle as P


def _plan(ctx, new, free, n_free, table, page=16, num_pages=100, T=None):
    T = sum(max(n, 0) for n in new) if T is None else T
    keep = np.full(T, -7, np.int32)
    return P.plan(ctx, new, np.array(free, np.int32), n_free, np.array(table, np.int32), page, num_pages, T, keep, keep)


def test_plan_by_hand():
    """Two sequences of 16-position pages: one at 14 cached positions adds 4 (two on its held page 7, two
    on a fresh one), one empty adds 17 (two fresh pages); the free list is used from its end."""
    r = _plan([14, 0], [4, 17], [3, 9, 50, 21], 4, [[7, -1, -1], [-1, -1, -1]], T=23)
    assert r["flags"] == 0 and r["n_free"] == 1
    assert r["q_start"].tolist() == [0, 4, 21] and r["kv_len"].tolist() == [18, 17]
    assert r["table"].tolist() == [[7, 21, -1], [50, 9, -1]]
    assert r["positions"].tolist() == [14, 15, 16, 17, *range(17), -7, -7]
    assert r["slots"].tolist() == [7 * 16 + 14, 7 * 16 + 15, 21 * 16, 21 * 16 + 1, *range(800, 816), 9 * 16, -7, -7]


def test_plan_errors_by_hand():
    assert _plan([16], [1], [], 0, [[5, -1]])["slots"].tolist() == [-1]              # free list exhausted
    r = _plan([31], [3], [4], 1, [[5, 6]])                                           # past the table's row
    assert r["flags"] == 16 and r["kv_len"].tolist() == [32] and r["slots"].tolist() == [6 * 16 + 15, -1, -1]
    r = _plan([-3, 2], [1, -1], [4], 1, [[5, 6], [7, -1]])                           # negative lengths
    assert r["flags"] == 16 and r["kv_len"].tolist() == [1, 2] and r["q_start"].tolist() == [0, 1, 1]
    r = _plan([0, 0], [3, 3], [4, 8], 2, [[-1], [-1]], T=4)                          # more tokens than rows
    assert r["flags"] == 16 and r["q_start"].tolist() == [0, 3, 4] and r["slots"].tolist() == [128, 129, 130, 64]
    assert _plan([3], [1], [], 0, [[100]])["slots"].tolist() == [-1]                 # a held page out of range


def test_append_by_hand():
    k = np.arange(1, 4, dtype=np.uint16).repeat(2).reshape(3, 2, 1)
    kc = np.zeros((2, 2, 4, 1), np.uint16)
    a, b, flags = P.append(k, k + 10, [6, -1, 9], 3, kc, kc)
    assert flags == 16 and a.sum() == 2 and a[1, :, 2, 0].tolist() == [1, 1] and b[1, 0, 2, 0] == 11
    assert P.append(k, k, [6, 1, 9], 2, kc, kc)[2] == 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (4, 0), (4, 2), (100, 3), (2, 100)])
def test_visible_by_enumeration(window, sinks):
    for p in range(-2, 12):
        want = [j for j in range(12) if j <= p and (window == 0 or j > p - window or j < sinks)]
        assert P.visible(p, 12, window, sinks).tolist() == want


def _paged(k, v, page, seed=0):
    """[H, N, D] keys and values -> shuffled pages and their table (NaN patterns behind the end)."""
    H, N, D = k.shape
    n = -(-N // page)
    order = np.random.default_rng(seed).permutation(n + 3)[:n]
    kc = np.full((n + 3, H, page, D), 0x7FC0, np.uint16)
    vc = kc.copy()
    for j in range(N):
        kc[order[j // page], :, j % page] = k[:, j]
        vc[order[j // page], :, j % page] = v[:, j]
    return kc, vc, order.astype(np.int32)[None]


def test_equals_the_contiguous_decode_oracle():
    inp = synth.make_attention(8, 2, 64, 50, seed=1)
    kc, vc, table = _paged(inp["k"], inp["v"], 16)
    o, mag, _ = P.attention(inp["q"][None], kc, vc, table, [0, 1], [50])
    assert np.allclose(o[0], A.gqa_decode_attention(inp["q"], inp["k"], inp["v"]), rtol=1e-12, atol=0)
    want = A.gqa_decode_attention(inp["q"], inp["k"], inp["v"] & np.uint16(0x7FFF))
    assert np.allclose(mag[0], want, rtol=1e-12, atol=0)


@pytest.mark.parametrize("window,sinks", [(0, 0), (7, 0), (7, 3)])
def test_chunk_rows_equal_single_tokens(window, sinks):
    """Row i of a chunk equals the decode oracle over the positions that it sees."""
    inp = synth.make_attention(4, 2, 64, 40, seed=2)
    q = synth.make_attention(9 * 4, 4, 64, 1, seed=3)["q"].reshape(9, 4, 64)
    kc, vc, table = _paged(inp["k"], inp["v"], 16)
    o, _, _ = P.attention(q, kc, vc, table, [0, 9], [40], window, sinks)
    for i in range(9):
        see = P.visible(31 + i, 40, window, sinks)
        assert np.allclose(o[i], A.gqa_decode_attention(q[i], inp["k"][:, see], inp["v"][:, see]), rtol=1e-12, atol=0)


def test_rows_before_position_zero_see_nothing():
    inp = synth.make_attention(2, 2, 64, 2, seed=4)
    kc, vc, table = _paged(inp["k"], inp["v"], 16)
    q = np.repeat(inp["q"][None], 3, 0)
    o, _, _ = P.attention(q, kc, vc, table, [0, 3], [2])
    assert (o[0] == 0).all() and np.allclose(o[1], P.to_f64(inp["v"][:, 0], "bf16")) and (o[2] != 0).any()


def test_fp16_patterns():
    assert P.to_f64(np.array([0x3C00, 0xC000, 0x3555], np.uint16), "fp16").tolist() == [1.0, -2.0, 1365 / 4096]
