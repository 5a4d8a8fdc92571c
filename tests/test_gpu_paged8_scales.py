"""Attention over the 8-bit paged cache where blocks' scales lie far apart: a row's result follows from what that row
sees, however large the scales of what other rows of its call see.

The bar is that of test_gpu_paged8.py with each term from the row's own visible positions: smax over positions whose weight is
not 0 in fp32 (above e^-80 of the row's largest; what lies below contributes nothing, however its score is rounded), and
the largest value that the row sees in place of the cache's.
"""
import math

import numpy as np
import pytest
import torch

import bit_quantized_expert_gb300 as moe
from oracle import paged8_oracle as Q
from oracle import paged_oracle as P
from test_gpu_paged import U, bits
from test_gpu_paged8 import Batch8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_quantized_expert_gb300 import build
    build.build()
    moe.load_library()


def by_row(b):
    """o and the parts of its bar in float64: o, sum of weight * |V|, smax, and the largest visible |V|, per row and head."""
    k_vals, v_vals = b.values()
    o, mag = (np.zeros((b.rows, b.Hq, b.D)) for _ in range(2))
    smax, vmax = (np.zeros((b.rows, b.Hq)) for _ in range(2))
    G = b.Hq // b.Hkv
    for i, (c, n) in enumerate(b.seqs):
        if n == 0:
            continue
        at, L = slice(b.q_start[i], b.q_start[i + 1]), c + n
        p, j = np.arange(c, L)[:, None], np.arange(L)[None, :]
        see = j <= p
        if b.window:
            see &= (j > p - b.window) | (j < b.sinks)
        for g in range(b.Hkv):
            kk, vv = Q.gather(k_vals, b.table[i], L, g), Q.gather(v_vals, b.table[i], L, g)
            for h in range(g * G, (g + 1) * G):
                qq = P.to_f64(b.q[at, h], b.dtype)
                s = np.where(see, qq @ kk.T / math.sqrt(b.D), -np.inf)
                s -= s.max(1, keepdims=True)
                e = np.exp(s)
                e /= e.sum(1, keepdims=True)
                o[at, h], mag[at, h] = e @ vv, e @ np.abs(vv)
                smax[at, h] = np.where(s > -80, np.abs(qq) @ np.abs(kk).T, 0.0).max(1) / math.sqrt(b.D)
                vmax[at, h] = np.where(see, np.abs(vv).max(1)[None, :], 0.0).max(1)
    return o, mag, smax, vmax


def check(b, label="", ref=None, want=0):
    ref, mag, smax, vmax = by_row(b) if ref is None else ref
    o, flags = b.run()
    assert flags == want, flags
    bad = np.isnan(ref)
    assert np.array_equal(np.isnan(o[:b.rows]), bad), label
    single = b.max_new == 1
    tol = U[b.dtype] * np.abs(ref) + mag * ((2.0 ** -17 if single else 2.0 ** -11) + 2.0 ** -18 +
                                            2 * smax[..., None] * (b.D // 16 + 4) * 2.0 ** -23)
    tol += int(b.kv_len.max()) * vmax[..., None] * (2.0 ** -39 if single else 2.0 ** -33)
    tol += 2.0 ** -25 if b.dtype == "fp16" else 0.0
    ratio = np.where(bad, 0.0, np.abs(o[:b.rows] - ref) / np.maximum(tol, 1e-300)).max((1, 2))
    print(f"{label}: max |o - ref| / bar = {ratio.max():.3f} in row {ratio.argmax()}")
    assert ratio.max() <= 1.0, (label, ratio.max(), np.flatnonzero(ratio > 1.0))


SPANS = (8, 14, 15, 16, 20, 24, 25, 31, 50, 66)
# (sequences, arguments, the block whose scale is far above the others'): rows before it, or behind its window, do not
# see it, others of their row block do
HIDDEN = [([(0, 60)], {}, 2), ([(700, 25)], {}, 44), ([(300, 100)], dict(window=64), 15), ([(0, 33), (6000, 40)], {}, 376),
          ([(100, 200)], dict(window=40, sinks=20), 12), ([(2072, 20)], dict(window=30), 127),
          ([(500, 20), (2070, 60)], dict(window=30, sinks=2), 128)]


@pytest.mark.parametrize("case", range(len(HIDDEN)))
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "fp16")])
def test_what_a_row_does_not_see_has_no_effect(case, which, D, dtype):
    """One block's keys or values 2^span above the others'."""
    seqs, kw, blk = HIDDEN[case]
    for span in SPANS:
        if which == 1 and dtype == "fp16" and span > 14:
            continue                            # past the type where it is seen
        b = Batch8(seqs, Hq=4, Hkv=2, D=D, dtype=dtype, page=32, seed=40 + case, spread=0, **kw)
        b.s[which][b.table[len(seqs) - 1, blk // 2], :, blk % 2] = 2.0 ** (span - 7)
        check(b, f"span {span}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_values_a_row_does_not_see_in_the_narrow_type(dtype):
    """As above with scales that stay within fp16: 2^span above 2^-20."""
    for seqs, kw, blk in HIDDEN:
        for span in (14, 16, 20, 25, 27):
            b = Batch8(seqs, Hq=8, Hkv=1, D=128, dtype=dtype, page=64, seed=50, **kw)
            b.s[1][:] = np.where(np.isnan(b.s[1]), np.nan, 2.0 ** -20)
            b.s[1][b.table[len(seqs) - 1, blk // 4], :, blk % 4] = 2.0 ** (span - 20)
            check(b, f"span {span}")


def test_values_a_row_does_not_see_at_the_ends_of_the_range():
    """Whole tiles of the largest scales that the first rows of the row block do not see, behind (or, of a window, before)
    tiles of the least ones."""
    for seqs, kw, first, last in (([(250, 20)], {}, 16, 17), ([(120, 100)], {}, 8, 14), ([(500, 110)], dict(window=130), 24, 31)):
        for low, high in ((-60, 60), (-60, 3), (-30, 60), (0, 60)):
            b = Batch8(seqs, Hq=4, Hkv=2, page=16, seed=51, **kw)
            b.s[1][:] = np.where(np.isnan(b.s[1]), np.nan, 2.0 ** low)
            for blk in range(first, min(last, -(-sum(seqs[0]) // 16))):
                b.s[1][b.table[0, blk]] = 2.0 ** high
            check(b, f"{low} {high}")


@pytest.mark.parametrize("new", [1, 25])
@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "fp16")])
def test_keys_beside_far_larger_ones(new, D, dtype):
    """One block of keys that all rows see, 2^span above the others' and pointing away from every query: it takes no part, and
    the scores of the others count as ever."""
    for seqs, blk in (([(100, new)], 3), ([(700, new)], 20), ([(700, new)], 0)):
        for span in SPANS:
            b = Batch8(seqs, Hq=4, Hkv=2, D=D, dtype=dtype, page=32, seed=60, spread=0, q_scale=0.5)
            b.q &= 0x7FFF
            page, off = b.table[0, blk // 2], blk % 2 * 16
            b.c[0][page, :, off:off + 16] = Q.to_codes(np.array(-448.0))
            b.s[0][page, :, blk % 2] = 2.0 ** (span - 7)
            check(b, f"span {span} at {blk}")


@pytest.mark.parametrize("seqs", [[(300, 70)], [(0, 130), (40, 1)], [(5000, 33)], [(500, 1), (20, 1)]])
@pytest.mark.parametrize("window", [0, 90])
def test_scales_at_random(seqs, window):
    """Any scales: of keys within what the scores allow, of values over their whole range."""
    for seed in range(4):
        b = Batch8(seqs, Hq=6, Hkv=3, D=64 if seed % 2 else 128, page=16, seed=70 + seed, window=window, q_scale=0.25)
        r = np.random.default_rng(seed)
        low = (-60, -40, -25, -12)[seed]
        b.s[0][:] = np.where(np.isnan(b.s[0]), np.nan, 2.0 ** r.integers(low, -5, b.s[0].shape))
        b.s[1][:] = np.where(np.isnan(b.s[1]), np.nan, 2.0 ** r.integers(*((-60, 61), (-30, 30), (-8, 8), (-60, -20))[seed], b.s[1].shape))
        check(b, f"seed {seed}")


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("span", [0, 20, 40])
def test_nan_in_a_block_of_far_larger_scale(which, span):
    """Rows that see the code have NaN (of a key everywhere, of a value in its dim), the others are not touched."""
    b = Batch8([(0, 60), (700, 25)], Hq=4, Hkv=2, page=32, seed=80, spread=0)
    for seq, blk in ((0, 2), (1, 44)):
        b.s[which][b.table[seq, blk // 2], :, blk % 2] = 2.0 ** (span - 7)
    ref = by_row(b)
    for seq, pos in ((0, 40), (1, 710)):
        b.c[which][b.table[seq, pos // 32], :, pos % 32, 5] = 0x7F
        c, n = b.seqs[seq]
        rows = slice(b.q_start[seq] + max(pos - c, 0), b.q_start[seq + 1])
        ref[0][rows, :, slice(None) if which == 0 else 5] = np.nan
    check(b, ref=ref, want=8)


@pytest.mark.parametrize("new", [1, 25])
@pytest.mark.parametrize("D", [64, 128])
def test_small_queries_beside_large_keys(new, D):
    """bf16 queries down to the least number under the largest key scale: keys point to and away from the query in turn, their
    values are 1 and -1, so that a result is the score's own size."""
    for size in (2.0 ** -46 * (1 + 2.0 ** -7), 2.0 ** -70, 2.0 ** -80 * (1 + 2.0 ** -7), 2.0 ** -84 * 1.5, 2.0 ** -86, 2.0 ** -100,
                 2.0 ** -133):
        b = Batch8([(64 - new, new)], Hq=4, Hkv=2, D=D, page=64, seed=90)
        page = b.table[0, 0]
        b.q[:] = bits(np.array(size), "bf16")
        sign = np.where(np.arange(64) % 2 == 0, 1.0, -1.0)[None, :, None]
        b.c[0][page], b.c[1][page] = Q.to_codes(448.0 * sign), Q.to_codes(sign)
        b.s[0][page], b.s[1][page] = 2.0 ** 60 if size < 2.0 ** -60 else 2.0 ** 36, 1.0
        check(b, f"size {size}")


@pytest.mark.parametrize("new", [1, 25])
@pytest.mark.parametrize("apart", [0, 30])
def test_least_queries_and_least_key_scales(new, apart):
    """Scores that are nothing beside 1: every visible value counts the same, what is masked does not count."""
    b = Batch8([(300, new), (0, new)], Hq=4, Hkv=2, page=32, seed=91, window=100, sinks=3)
    b.q[:] = bits(np.array(2.0 ** -126), "bf16")
    for i, low in ((0, -60), (1, -20)):
        b.s[i][:] = np.where(np.isnan(b.s[i]), np.nan, 2.0 ** low)
        b.s[i][b.table[0, 9], :, 1] = 2.0 ** (low + apart)
    check(b)


@pytest.mark.parametrize("new", [1, 45])
def test_repeats_and_graphs(new):
    """Blocks of far larger scale among others: the same bits every time, beside another batch, and from a graph."""
    batches = []
    for seed in (0, 1):
        b = Batch8([(3000, new), (40, new), (0, new)], Hq=8, Hkv=2, seed=95 + seed)
        r = np.random.default_rng(seed)
        for i in range(2):
            up = r.random(b.s[i].shape) < 0.02
            b.s[i][up] *= 2.0 ** 25
        b.upload()
        b.attend()
        batches.append(b)
    first = [b.dev["o"].clone() for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, b in zip(streams, batches):
            b.attend(stream=s)
    torch.cuda.synchronize()
    for b, want in zip(batches, first):
        assert torch.equal(b.dev["o"], want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.attend()
        b.dev["o"].zero_()
        g.replay()
        assert torch.equal(b.dev["o"], want) and b.flags() == 0
