"""The paged key/value cache on the GPU against the oracle: plan and append exactly, attention within a
bar that follows from its arithmetic.

Bar per output element, with u = 2^-8 (bf16) or 2^-11 (fp16), half a step of the type:
  u * |ref|                      the one rounding of the output;
  u_p * mag                      rounding of the softmax numerators before the product with V: u in the
                                 chunk form, 2^-17 in the single-token form, which keeps the remainders
                                 (fp16 pairs hold at least as much);
  2 * smax * (D/16 + 2) * 2^-23 * mag   the scores: D/16 tensor-core steps and two fp32 roundings, each
                                 within 2^-23 (an accumulator that truncates) of sum_i |q_i k_i| / sqrt(D)
                                 <= smax, moving a numerator by that fraction (the factor 2 also covers
                                 its denominator; log2(e) and ln 2 cancel);
  2^-19 * mag                    exp2 (2 ulp), the running sums and rescales in fp32, the merge: a few
                                 dozen steps of 2^-24;
  fp16 only, 2^-25 * (1 + N max|V|)   subnormal outputs, and numerators below 2^-14, held to 2^-25.
mag is the same attention over |V|.
"""
import numpy as np
import pytest
import torch

import bit_quantized_expert_gb300 as moe
from oracle import paged_oracle as P

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}
NAN = {"bf16": 0x7FC1, "fp16": 0x7E01}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_quantized_expert_gb300 import build
    build.build()
    moe.load_library()


def bits(x, dtype):
    """float32 array -> 16-bit patterns, rounded to nearest."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(TORCH[dtype]).view(torch.int16).numpy().view(np.uint16)


def dev(a, dtype=None):
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        t = torch.from_numpy(a.view(np.int16)).cuda()
        return t if dtype is None else t.view(TORCH[dtype])
    return torch.from_numpy(a.astype(np.int32)).cuda()


def host(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class Batch:
    """Sequences with (cached, new) positions in shuffled pages.  Whatever no sequence wrote is NaN."""

    def __init__(self, seqs, Hq=16, Hkv=2, D=128, page=64, dtype="bf16", layout="head", fused=False, pad=0, window=0,
                 sinks=0, seed=0, q_scale=1.0, max_new=None, extra_pages=3):
        r = np.random.default_rng(seed)
        self.seqs, self.Hq, self.Hkv, self.D, self.page, self.dtype = seqs, Hq, Hkv, D, page, dtype
        self.window, self.sinks, self.layout = window, sinks, layout
        B, rows = len(seqs), sum(n for _, n in seqs)
        T = rows + pad
        kv = [c + n for c, n in seqs]
        need = [-(-x // page) for x in kv]
        self.P, self.M = sum(need) + extra_pages, max(need + [1]) + 1
        order = r.permutation(self.P)
        self.table = np.full((B, self.M), -1, np.int32)
        at = 0
        kc = np.full((self.P, Hkv, page, D), NAN[dtype], np.uint16)
        vc = kc.copy()
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            k = bits(r.standard_normal((need[b], Hkv, page, D)), dtype)
            v = bits(r.standard_normal((need[b], Hkv, page, D)), dtype)
            live = (np.arange(need[b] * page) < kv[b]).reshape(-1, 1, page, 1)
            kc[self.table[b, :need[b]]] = np.where(live, k, NAN[dtype])
            vc[self.table[b, :need[b]]] = np.where(live, v, NAN[dtype])
        self.kc, self.vc = kc, vc
        self.q = bits(r.standard_normal((T, Hq, D)) * q_scale, dtype)
        self.k, self.v = (bits(r.standard_normal((T, Hkv, D)), dtype) for _ in range(2))
        self.q_start = np.cumsum([0] + [n for _, n in seqs]).astype(np.int32)
        self.kv_len = np.array(kv, np.int32)
        self.T, self.rows, self.fused = T, rows, fused
        self.max_new = max([n for _, n in seqs] + [1]) if max_new is None else max_new

    def upload(self):
        d = self.dtype
        kc, vc = dev(self.kc, d), dev(self.vc, d)
        if self.layout == "position":
            kc, vc = (c.transpose(1, 2).contiguous().transpose(1, 2) for c in (kc, vc))
        elif self.layout == "interleaved":
            both = torch.stack([kc, vc], 1)
            kc, vc = both[:, 0], both[:, 1]
        q, k, v = dev(self.q, d), dev(self.k, d), dev(self.v, d)
        if self.fused:
            x = torch.cat([t.reshape(self.T, -1) for t in (q, k, v)], 1)
            q, k, v = (t.view(self.T, -1, self.D) for t in x.split([t.shape[1] * self.D for t in (q, k, v)], 1))
        o_wide = torch.full((self.T, self.Hq * self.D + (64 if self.fused else 0)), 7.0, dtype=TORCH[d], device="cuda")
        o = o_wide[:, :self.Hq * self.D].view(self.T, self.Hq, self.D)
        self.dims = moe.gqa_paged_dims(self.Hq, self.Hkv, self.D, self.page, self.P, self.M, len(self.seqs), self.T,
                                       max_new=self.max_new, window=self.window, sinks=self.sinks, dtype=d,
                                       q_stride=q.stride(0), k_stride=k.stride(0), v_stride=v.stride(0),
                                       o_stride=o.stride(0), cache_strides=kc.stride()[:3])
        self.dev = dict(q=q, k=k, v=v, kc=kc, vc=vc, o=o, o_wide=o_wide, table=dev(self.table), q_start=dev(self.q_start),
                        kv_len=dev(self.kv_len), ws=moe.alloc_gqa_paged_workspace(self.dims))
        return self.dev

    def attend(self, stream=None):
        x = self.dev
        moe.gqa_paged_attention(self.dims, x["q"], x["kc"], x["vc"], x["table"], x["q_start"], x["kv_len"], x["o"], x["ws"],
                                stream=stream)

    def run(self):
        self.upload()
        self.attend()
        return P.to_f64(host(self.dev["o"]), self.dtype), moe.read_error_flags(self.dev["ws"])

    def oracle(self, kc=None, vc=None):
        return P.attention(self.q, self.kc if kc is None else kc, self.vc if vc is None else vc, self.table, self.q_start,
                           self.kv_len, self.window, self.sinks, self.dtype)

    def check(self, o, ref=None, rows=None, label=""):
        ref, mag, smax = self.oracle() if ref is None else ref
        rows = np.arange(self.rows) if rows is None else rows
        u, n = U[self.dtype], int(self.kv_len.max())
        u_p = 2.0 ** -17 if self.max_new == 1 else u
        tol = u * np.abs(ref) + mag * (u_p + 2.0 ** -19 + 2 * smax[..., None] * (self.D // 16 + 2) * 2.0 ** -23)
        if self.dtype == "fp16":
            vmax = np.abs(np.nan_to_num(P.to_f64(self.vc, "fp16"), nan=0.0, posinf=0.0, neginf=0.0)).max()
            tol = tol + 2.0 ** -25 * (1 + n * vmax)
        ratio = (np.abs(o - ref)[rows] / np.maximum(tol[rows], 1e-30)).max() if len(rows) else 0.0
        print(f"{label}: max |o - ref| / bar = {ratio:.3f}")
        assert ratio <= 1.0, (label, ratio)
        # rows behind the last sequence, and what lies between the rows of a wider buffer
        assert (o[self.rows:] == 7.0).all()
        assert (self.dev["o_wide"][:, self.Hq * self.D:].float() == 7.0).all()


def _ok(batch, label=""):
    o, flags = batch.run()
    assert flags == 0, flags
    batch.check(o, label=label)
    return o


# ---------------------------------------------------------------- attention: single tokens
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_single_tokens_ragged(dtype, page):
    ctx = [0, 1, 14, 15, 16, 62, 63, 64, 65, 127, 128, 200, 511, 1000, 2049]
    _ok(Batch([(c, 1) for c in ctx], page=page, dtype=dtype, seed=page), f"{dtype} page {page}")


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 8, 128), (6, 2, 128), (5, 1, 64), (32, 4, 128), (7, 7, 64), (14, 2, 64), (1, 1, 128),
                                      (24, 3, 64)])
def test_single_tokens_head_layouts(Hq, Hkv, D):
    _ok(Batch([(c, 1) for c in (0, 77, 300, 640)], Hq=Hq, Hkv=Hkv, D=D, page=32, seed=Hq), f"{Hq}/{Hkv} D {D}")


@pytest.mark.parametrize("layout", ["position", "interleaved"])
@pytest.mark.parametrize("D", [64, 128])
def test_single_tokens_strides(layout, D):
    _ok(Batch([(c, 1) for c in (3, 90, 257)], D=D, layout=layout, fused=True, pad=5, dtype="fp16", page=16, seed=9), layout)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 0), (100, 4), (100, 70), (129, 300), (4000, 4)])
def test_single_tokens_window(window, sinks):
    _ok(Batch([(c, 1) for c in (0, 1, 63, 99, 100, 163, 500, 1500)], window=window, sinks=sinks, page=16, seed=3),
        f"window {window} sinks {sinks}")


def test_single_tokens_idle_sequences_and_padding():
    """Sequences without a new token between others; rows behind the last one stay as they were."""
    _ok(Batch([(70, 0), (5, 1), (0, 0), (130, 1), (64, 0)], max_new=1, pad=3, seed=4))


def test_single_tokens_long_and_short_together():
    _ok(Batch([(20000, 1)] + [(c, 1) for c in range(0, 90, 3)] + [(9000, 1)], Hq=8, Hkv=2, seed=5))


def test_single_tokens_many_sequences():
    _ok(Batch([(c % 23, 1) for c in range(1500)], Hq=2, Hkv=1, D=64, page=16, dtype="fp16", seed=6))


@pytest.mark.parametrize("q_scale", [8.0, 0.01])
def test_single_tokens_peaked_and_flat(q_scale):
    _ok(Batch([(3000, 1), (100, 1)], q_scale=q_scale, seed=7))


# ---------------------------------------------------------------- attention: chunks
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_chunks_ragged(dtype, page):
    seqs = [(0, 2), (0, 1), (0, 17), (5, 33), (127, 1), (128, 2), (100, 64), (300, 31), (0, 130), (513, 5)]
    _ok(Batch(seqs, Hq=8, Hkv=1, page=page, dtype=dtype, seed=page), f"{dtype} page {page}")


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 4, 128), (6, 2, 128), (5, 1, 64), (16, 4, 64), (3, 3, 64), (14, 2, 128), (1, 1, 128),
                                      (12, 2, 64)])
def test_chunks_head_layouts(Hq, Hkv, D):
    _ok(Batch([(0, 70), (200, 45), (37, 1)], Hq=Hq, Hkv=Hkv, D=D, page=32, seed=Hq), f"{Hq}/{Hkv} D {D}")


@pytest.mark.parametrize("layout", ["position", "interleaved"])
@pytest.mark.parametrize("D", [64, 128])
def test_chunks_strides(layout, D):
    _ok(Batch([(3, 40), (90, 3), (140, 20)], Hq=8, D=D, layout=layout, fused=True, pad=5, dtype="fp16", page=16, seed=9), layout)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (100, 4), (100, 200), (128, 0), (300, 130), (4000, 4)])
def test_chunks_window(window, sinks):
    _ok(Batch([(0, 150), (400, 70), (1000, 9)], Hq=8, Hkv=2, window=window, sinks=sinks, page=16, seed=3),
        f"window {window} sinks {sinks}")


def test_chunks_idle_sequences_and_padding():
    _ok(Batch([(70, 0), (5, 20), (0, 0), (130, 1), (64, 0)], pad=130, seed=4))


def test_chunk_over_a_long_cache():
    _ok(Batch([(6000, 9), (0, 3), (3000, 20)], Hq=4, Hkv=2, seed=5))


@pytest.mark.parametrize("seqs,Hq,Hkv,D", [([(20000, 3)], 8, 1, 128), ([(9000, 40)], 4, 2, 64), ([(6000, 33)], 16, 2, 128),
                                           ([(30000, 2), (50, 4), (7000, 17)], 6, 1, 64)])
def test_few_rows_over_long_caches(seqs, Hq, Hkv, D):
    """Items cut into many parts (up to one a SM), of one row tile and of two."""
    _ok(Batch(seqs, Hq=Hq, Hkv=Hkv, D=D, seed=29))


@pytest.mark.parametrize("q_scale", [8.0, 0.01])
def test_chunks_peaked_and_flat(q_scale):
    _ok(Batch([(1000, 40), (100, 30)], Hq=8, q_scale=q_scale, seed=7))


def test_scores_that_grow_along_the_cache():
    """Every key is a larger multiple of the query than the one before it: the running maximum moves at
    every tile, so everything summed before is scaled down again and again."""
    for new, hq in ((1, 8), (30, 2)):
        b = Batch([(900, new)], Hq=hq, Hkv=1, seed=8, q_scale=0.5)
        q = P.to_f64(b.q[0, 0], "bf16")
        flat = np.arange(900 + new)
        k = bits(np.outer((flat + 1) / 60.0, q), "bf16")
        for j in flat:
            b.kc[b.table[0, j // 64], 0, j % 64] = k[j]
        b.q[:] = b.q[0, 0]
        _ok(b, f"new {new}")


@pytest.mark.parametrize("new", [1, 20])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_weight_spread_over_tiny_numerators(new, dtype):
    """One position e^18 above all others, which alone have values: fp16 holds no number as small as e^-18, so
    the numerators have to use its range from 2^15 down.  160 sequences over the same pages, so that a share
    is about one of them.  Bar as above, but with numerators held to 2^-25 of 2^-9 (chunks) or of 2^-15
    (single tokens) of the row's largest."""
    b = Batch([(16384 - new, new)], Hq=1, Hkv=1, D=64, page=128, dtype=dtype, seed=28)
    one = bits(np.ones(1), dtype)[0]
    b.q[:], b.kc[b.table[0, :128]], b.vc[b.table[0, :128]] = 0, 0, one
    b.q[:, 0, 0], b.kc[b.table[0, 0], 0, 0, 0] = bits(np.array([8.0, 18.0]), dtype)
    b.vc[b.table[0, 0], 0, 0] = 0
    ref, mag, smax = b.oracle()
    n = 160
    b.table, b.q, b.kv_len = np.repeat(b.table, n, 0), np.tile(b.q, (n, 1, 1)), np.repeat(b.kv_len, n)
    b.k, b.v = (np.tile(x, (n, 1, 1)) for x in (b.k, b.v))
    b.q_start, b.seqs = (np.arange(n + 1) * new).astype(np.int32), b.seqs * n
    b.T = b.rows = n * new
    o, flags = b.run()
    assert flags == 0
    u = U[dtype]
    tol = u * np.abs(ref) + mag * ((2.0 ** -17 if new == 1 else u) + 2.0 ** -19 + 2 * smax[..., None] * 6 * 2.0 ** -23)
    if dtype == "fp16":
        tol = tol + 2.0 ** -25 * (1 + 16384 * 2.0 ** (-15 if new == 1 else -9))
    ratio = (np.abs(o.reshape(n, new, 1, 64) - ref) / tol).max()
    print(f"{dtype}, {new} new: max |o - ref| / bar = {ratio:.3f}")
    assert ratio <= 1.0


# ---------------------------------------------------------------- what a row does not see
def _slot(b, s, p):
    return b.table[s, p // b.page], p % b.page


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", [0x7F80, 0xFF80, 0x7FC0], ids=["inf", "-inf", "nan"])
def test_non_finite_values_reach_only_rows_that_see_them(value, D):
    """One value and one key of a chunk's own new positions: earlier rows do not see them."""
    b = Batch([(50, 40), (0, 12)], Hq=8, D=D, page=16, seed=11)
    clean = b.oracle()
    pv, pk = _slot(b, 0, 50 + 25), _slot(b, 0, 50 + 33)
    b.vc[pv[0], 1, pv[1], 17] = value
    b.kc[pk[0], 0, pk[1], 5] = value
    o, flags = b.run()
    assert flags == moe.ERR_NON_FINITE
    heads = b.Hq // 2
    for row in range(40):
        if row < 33:
            b.check(o[:, :heads], tuple(x[:, :heads] for x in clean), [row])
        if row < 25:
            b.check(o[:, heads:], tuple(x[:, heads:] for x in clean), [row])
        else:
            assert not np.isfinite(o[row, heads:, 17]).any()
            if value == 0x7F80:
                assert (o[row, heads:, 17] == np.inf).all()
            other = np.arange(D) != 17
            b.check(o[:, heads:][:, :, other], tuple(x[:, heads:][:, :, other] if x.ndim == 3 else x[:, heads:] for x in clean),
                    [row])
    b.check(o, clean, np.arange(40, 52))


@pytest.mark.parametrize("new", [1, 30])
def test_passed_window_pages_hold_anything(new):
    """Positions behind the window are NaN and their wholly passed pages are gone from the table."""
    b = Batch([(500, new), (90, new)], window=100, sinks=5, page=16, Hq=8, seed=12)
    clean = b.oracle()
    for s, (c, n) in enumerate(b.seqs):
        lo = max(c - 99, 0)
        for p in range(5, lo):
            at = _slot(b, s, p)
            b.kc[at[0], :, at[1]] = b.vc[at[0], :, at[1]] = NAN["bf16"]
        for i in range(1, lo // 16):
            b.table[s, i] = 1 << 30
    o, flags = b.run()
    assert flags == 0
    b.check(o, clean)


def test_rows_that_see_nothing_are_zero():
    """More new tokens than positions: the rows before position 0 are zeros."""
    b = Batch([(0, 30), (9, 1)], Hq=8, seed=13)
    b.kv_len[0] = 12
    o, flags = b.run()
    assert flags == 0 and (o[:18] == 0).all()
    b.check(o)
    b = Batch([(0, 30)], Hq=8, seed=13)
    b.kv_len[0] = 0
    o, flags = b.run()
    assert flags == 0 and (o == 0).all()
    b = Batch([(0, 1), (9, 1)], seed=13)
    b.kv_len[0] = 0
    o, flags = b.run()
    assert flags == 0 and (o[0] == 0).all()
    b.check(o)


# ---------------------------------------------------------------- out of range, without a fault
@pytest.mark.parametrize("new", [1, 20])
@pytest.mark.parametrize("page_no", [-1, -5, 10**6, 2**31 - 1, -2**31])
def test_bad_pages_count_as_zeros(new, page_no):
    b = Batch([(150, new), (90, new)], Hq=8, page=32, seed=14)
    b.table[0, 2] = page_no
    o, flags = b.run()
    assert flags == moe.ERR_BAD_PAGES
    b.check(o)


@pytest.mark.parametrize("new", [1, 20])
def test_lengths_out_of_range(new):
    """kv_len above the block-table row or negative, q_start that falls or passes T: bit 16, the other
    sequences as they are."""
    for change in ("long", "negative", "falls", "passes"):
        b = Batch([(150, new), (90, new), (30, new)], Hq=8, page=32, seed=15)
        clean = b.oracle()
        rows = np.arange(new, 2 * new) if change in ("long", "negative") else np.arange(new)
        if change == "long":
            b.kv_len[0] = 10**9
        elif change == "negative":
            b.kv_len[0] = -4
        elif change == "falls":
            b.q_start[2] = -7
        else:
            b.q_start[2:] = 10**8
        o, flags = b.run()
        assert flags & moe.ERR_BAD_PAGES, change
        b.check(o, clean, rows, change)


@pytest.mark.parametrize("new", [1, 2])
def test_more_work_than_can_be_numbered(new):
    """Lengths whose cache tiles pass 2^32 over all sequences and heads (every other sequence claims the same
    rows, each over 2^30 positions): flagged, and nothing is computed."""
    B, H, page, M = 132, 8, 128, 1 << 23
    d = moe.gqa_paged_dims(H, H, 64, page, 4, M, B, new, max_new=new)
    i32 = dict(dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(4, H, page, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, o = torch.ones(new, H, 64, dtype=torch.bfloat16, device="cuda"), torch.full((new, H, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    table, kv = torch.zeros(B, M, **i32), torch.full((B,), M * page, **i32)
    starts, ws = torch.arange(B + 1, **i32) % 2 * new, moe.alloc_gqa_paged_workspace(d)
    assert B // 2 * H * (M * page // (64 if new == 1 else 128)) >= 2 ** 32
    moe.gqa_paged_attention(d, q, kc, vc, table, starts.int(), kv, o, ws)
    assert moe.read_error_flags(ws) == moe.ERR_BAD_PAGES and (o == 7.0).all()


def test_more_rows_than_max_new():
    """The first max_new rows of the sequence are computed, the rest left as they were."""
    for limit in (1, 5):
        b = Batch([(20, 8), (30, 1)], Hq=8, seed=16, max_new=limit)
        o, flags = b.run()
        assert flags == moe.ERR_BAD_PAGES
        b.check(o, rows=np.r_[0:limit, 8])
        assert (o[limit:8] == 7.0).all()


def test_offsets_beyond_32_bits():
    """Pages whose elements lie past 2^31 and past 2^32 of a cache of 9 GB a tensor."""
    page, H, D = 128, 2, 128
    num = (1 << 32) // (page * H * D) + 5000
    kc = torch.empty((num, H, page, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    pages = [num - 1, 65536, 65535, num - 4000, 131071, 131072]
    gen = torch.Generator(device="cuda").manual_seed(3)
    for p in pages:
        for c in (kc, vc):
            c[p].copy_(torch.randn((H, page, D), device="cuda", generator=gen))
    small = [host(torch.stack([c[p] for p in pages])) for c in (kc, vc)]
    table = torch.tensor([pages + [-1]], dtype=torch.int32, device="cuda")
    for new in (1, 20):
        b = Batch([(700 - new, new)], Hq=8, Hkv=H, page=page, seed=17)
        b.upload()
        b.kc, b.vc, b.table = small[0], small[1], np.arange(6, dtype=np.int32)[None]
        d = moe.gqa_paged_dims(8, H, D, page, num, 7, 1, new, max_new=new)
        ws = moe.alloc_gqa_paged_workspace(d)
        moe.gqa_paged_attention(d, b.dev["q"], kc, vc, table, b.dev["q_start"], b.dev["kv_len"], b.dev["o"], ws)
        assert moe.read_error_flags(ws) == 0
        b.check(P.to_f64(host(b.dev["o"]), "bf16"), label=f"new {new}")
        slots = torch.tensor([pages[0] * page + 5 + i for i in range(new)], dtype=torch.int32, device="cuda")
        moe.gqa_paged_append(d, b.dev["k"], b.dev["v"], slots, b.dev["q_start"], kc, vc, ws)
        assert (host(kc[pages[0]])[:, 5:5 + new] == b.k.transpose(1, 0, 2)).all()
        kc[pages[0]].copy_(dev(small[0][0], "bf16"))
        vc[pages[0]].copy_(dev(small[1][0], "bf16"))


# ---------------------------------------------------------------- calls in company
@pytest.mark.parametrize("new", [1, 150])
def test_identical_across_calls(new):
    b = Batch([(5000, new), (10, new), (777, new)], Hq=8, seed=18)
    first, _ = b.run()
    for _ in range(5):
        b.dev["o"].fill_(7.0)
        b.attend()
        assert np.array_equal(P.to_f64(host(b.dev["o"]), "bf16"), first)


def test_two_calls_at_once_on_two_streams():
    """Chunks on one stream beside single tokens on another, each with its own workspace."""
    a, b = Batch([(900, 200), (50, 30)], Hq=8, seed=19), Batch([(4000, 1), (3, 1)], Hq=8, seed=20)
    ra, rb = a.run()[0], b.run()[0]
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (sa, sb):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        a.attend(stream=sa)
        b.attend(stream=sb.cuda_stream)
    torch.cuda.synchronize()
    assert np.array_equal(P.to_f64(host(a.dev["o"]), "bf16"), ra) and np.array_equal(P.to_f64(host(b.dev["o"]), "bf16"), rb)


def test_binding_refuses_what_does_not_fit():
    """Wrong types, shapes, strides, contiguity and host tensors raise before anything is launched."""
    b = Batch([(20, 3), (5, 1)], seed=21)
    x = b.upload()
    good = dict(q=x["q"], k_cache=x["kc"], v_cache=x["vc"], block_table=x["table"], q_start=x["q_start"], kv_len=x["kv_len"],
                o=x["o"], workspace=x["ws"])
    wide = torch.zeros((4, 16, 256), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(q=x["q"].to(torch.float16)), dict(q=x["q"].float()), dict(q=x["q"][:3]), dict(q=x["q"].cpu()),
                dict(q=wide[:, :, :128]), dict(o=x["o"].view(4, 2048)), dict(k_cache=x["kc"].transpose(1, 2)),
                dict(v_cache=x["vc"][1:]), dict(k_cache=x["kc"].half(), v_cache=x["vc"].half()),
                dict(block_table=x["table"].long()), dict(block_table=x["table"][:1]), dict(q_start=x["q_start"][1:]),
                dict(kv_len=x["kv_len"].float()), dict(kv_len=x["kv_len"].cpu()), dict(workspace=x["ws"].cpu())):
        with pytest.raises(ValueError):
            moe.gqa_paged_attention(b.dims, **{**good, **bad})
    with pytest.raises(moe.MoeError):
        moe.gqa_paged_attention(b.dims, **{**good, "workspace": x["ws"][:-256]})
    # bit patterns are as good as the type
    moe.gqa_paged_attention(b.dims, **{**good, "q": x["q"].view(torch.int16), "o": x["o"].view(torch.int16)})
    b.check(P.to_f64(host(x["o"]), "bf16"))


def test_nothing_to_do_on_the_gpu():
    """No tokens: nothing is launched or written; no sequence with rows: nothing is written."""
    b = Batch([(20, 0), (5, 0)], pad=4, seed=22)
    o, flags = b.run()
    assert flags == 0 and (o == 7.0).all()
    b.max_new = 1
    o, flags = b.run()
    assert flags == 0 and (o == 7.0).all()
    d = moe.gqa_paged_dims(16, 2, 128, 64, b.P, b.M, 2, 0)
    z = torch.zeros((0, 16, 128), dtype=torch.bfloat16, device="cuda")
    x = b.dev
    moe.gqa_paged_attention(d, z, x["kc"], x["vc"], x["table"], x["q_start"], x["kv_len"], z, moe.alloc_gqa_paged_workspace(d))


def test_many_short_chunks():
    """More row blocks than one warp schedules: the block makes the schedule (300 and 4096 sequences)."""
    r = np.random.default_rng(23)
    _ok(Batch([(int(c), int(n)) for c, n in zip(r.integers(0, 200, 300), r.integers(0, 12, 300))], Hq=4, Hkv=1, D=64, page=16,
              seed=23), "300 sequences")
    _ok(Batch([(int(c), int(n)) for c, n in zip(r.integers(0, 20, 4096), r.integers(0, 3, 4096))], Hq=2, Hkv=1, D=64, page=16,
              seed=24, max_new=2), "4096 sequences")
    _ok(Batch([(int(c), 1) for c in r.integers(0, 40, 4096)], Hq=2, Hkv=2, D=64, page=16, seed=25), "4096 single tokens")


def test_one_long_prompt():
    """Thousands of new tokens of one sequence with nothing cached: row blocks of 1 to 9 tiles, many of them
    whole in a share, checked on every 13th row."""
    b = Batch([(0, 1200)], Hq=4, Hkv=1, seed=26)
    o, flags = b.run()
    assert flags == 0
    rows = np.arange(0, 1200, 13)
    sub = Batch([(0, 1200)], Hq=4, Hkv=1, seed=26)
    ref, mag, smax = (np.zeros((1200, 4, 128)), np.zeros((1200, 4, 128)), np.zeros((1200, 4)))
    for t in rows:
        one = P.attention(sub.q[t:t + 1], sub.kc, sub.vc, sub.table, [0, 1], [t + 1])
        ref[t], mag[t], smax[t] = one[0][0], one[1][0], one[2][0]
    b.check(o, (ref, mag, smax), rows)


def test_sequences_that_share_pages():
    """Two sequences whose tables name the same pages (a common prompt)."""
    for new in (1, 12):
        b = Batch([(100, new), (96, new)], Hq=8, page=32, seed=27)
        b.table[1, :3] = b.table[0, :3]
        _ok(b, f"new {new}")


# ---------------------------------------------------------------- plan
def _plan_case(ctx, new, page, num_pages, M, pad, seed, n_free=None, table=None):
    r = np.random.default_rng(seed)
    order = r.permutation(num_pages).astype(np.int32)
    tab = np.full((len(ctx), M), -9, np.int32)
    at = 0
    for b, c in enumerate(ctx):
        n = -(-max(0, min(c, M * page)) // page)
        tab[b, :n] = order[at:at + n]
        at += n
    free = order[at:]
    T = sum(max(0, n) for n in new) + pad
    return dict(ctx=ctx, new=new, free=free, n_free=len(free) if n_free is None else n_free, table=tab, page=page,
                num_pages=num_pages, T=T)


def _plan_run(c, in_place=True, positions=True, T=None):
    T = c["T"] if T is None else T
    B, M = c["table"].shape
    d = moe.gqa_paged_dims(16, 2, 128, c["page"], c["num_pages"], M, B, T)
    ws = moe.alloc_gqa_paged_workspace(d)
    i32 = dict(dtype=torch.int32, device="cuda")
    t = dict(table=dev(c["table"]), q_start=torch.full((B + 3,), -7, **i32), kv_len=torch.full((B + 3,), -7, **i32),
             positions=torch.full((T + 3,), -7, **i32), slots=torch.full((T + 3,), -7, **i32), n_free=dev(np.array([c["n_free"]])))
    out = t["n_free"] if in_place else torch.zeros(1, **i32)
    free = dev(c["free"]) if len(c["free"]) else torch.zeros(1, **i32)[:0]
    moe.gqa_paged_plan(d, dev(np.array(c["ctx"])), dev(np.array(c["new"])), free, t["n_free"], t["table"], t["q_start"],
                       t["kv_len"], t["positions"] if positions else None, t["slots"], out, ws)
    flags = moe.read_error_flags(ws)
    got = {k: v.cpu().numpy() for k, v in t.items()}
    got["n_free"] = int(out[0])
    keep = np.full(T, -7, np.int32)
    want = P.plan(c["ctx"], c["new"], c["free"], c["n_free"], c["table"], c["page"], c["num_pages"], T, keep, keep)
    assert flags == want["flags"]
    assert np.array_equal(got["table"], want["table"])
    assert got["n_free"] == want["n_free"]
    assert np.array_equal(got["q_start"][:B + 1], want["q_start"]) and (got["q_start"][B + 1:] == -7).all()
    assert np.array_equal(got["kv_len"][:B], want["kv_len"]) and (got["kv_len"][B:] == -7).all()
    assert np.array_equal(got["slots"][:T], want["slots"]) and (got["slots"][T:] == -7).all()
    if positions:
        assert np.array_equal(got["positions"][:T], want["positions"]) and (got["positions"][T:] == -7).all()
    return want


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("B", [1, 2, 33, 300, 1025, 4096])
def test_plan(B, page):
    r = np.random.default_rng(B + page)
    ctx = [int(x) for x in r.integers(0, 5 * page, B)]
    new = [int(x) for x in r.choice([0, 1, 1, 1, 2, page, page + 1, 3 * page], B)]
    num = sum(-(-(c + n) // page) for c, n in zip(ctx, new)) + 5
    want = _plan_run(_plan_case(ctx, new, page, num, 9, 7, B), in_place=bool(B % 2))
    assert want["flags"] == 0


def test_plan_sizes_at_the_ends():
    _plan_run(_plan_case([0], [0], 16, 4, 3, 5, 1))                              # nothing new at all
    _plan_run(_plan_case([0, 3], [0, 0], 16, 4, 3, 0, 1))                        # T = 0
    _plan_run(_plan_case([0], [70000], 64, 1200, 1100, 0, 1), positions=False)   # one long prompt
    _plan_run(_plan_case([15, 16, 17] * 50, [1, 1, 1] * 50, 16, 400, 3, 0, 1))   # decode across page ends
    _plan_run(_plan_case([48] * 4, [0] * 4, 16, 12, 3, 0, 1))                    # full rows, no free page


def test_plan_without_rows():
    """T = 0 with empty tensors for the tokens and the free list (whose pointers are null)."""
    d = moe.gqa_paged_dims(4, 2, 64, 16, 8, 3, 2, 0)
    i32 = dict(dtype=torch.int32, device="cuda")
    ws, none = moe.alloc_gqa_paged_workspace(d), torch.zeros(0, **i32)
    ctx, table, free = torch.tensor([5, 0], **i32), torch.full((2, 3), 4, **i32), torch.zeros(1, **i32)
    starts, kv = torch.full((3,), 9, **i32), torch.full((2,), 9, **i32)
    moe.gqa_paged_plan(d, ctx, torch.zeros(2, **i32), none, free, table, starts, kv, none, none, free, ws)
    assert starts.tolist() == [0, 0, 0] and kv.tolist() == [5, 0] and free.item() == 0 and (table == 4).all()
    assert moe.read_error_flags(ws) == 0
    with pytest.raises(moe.MoeError):   # lengths updated in place: refused
        moe.gqa_paged_plan(d, ctx, torch.zeros(2, **i32), none, free, table, starts, ctx, none, none, free, ws)


@pytest.mark.parametrize("what", ["exhausted", "empty", "over_row", "over_T", "negative", "bad_free", "bad_held", "n_free_high",
                                  "n_free_negative", "huge"])
def test_plan_out_of_range(what):
    ctx, new, page, M, T = [10, 40, 0, 31, 16], [30, 1, 17, 2, 0], 16, 5, None
    c = _plan_case(ctx, new, page, 30, M, 3, 5)
    if what == "exhausted":
        c["n_free"] = 2
    elif what == "empty":
        c["free"], c["n_free"] = c["free"][:0], 0
    elif what == "over_row":
        c["new"] = [30, 60, 17, 2, 0]
        c["T"] += 59
    elif what == "over_T":
        T = 40
    elif what == "negative":
        c["ctx"], c["new"] = [10, -40, 0, 31, 16], [30, 1, 17, -2, 0]
    elif what == "bad_free":
        c["free"][-2], c["free"][-4] = 30, -1
    elif what == "bad_held":
        c["table"][0, 0], c["table"][3, 1] = 77, -3
    elif what == "n_free_high":
        c["n_free"] = len(c["free"]) + 1
    elif what == "n_free_negative":
        c["n_free"] = -3
    else:
        c["ctx"], c["new"] = [2**31 - 1, 0, 0, 0, 2**31 - 1], [2**31 - 1] * 5
        T = 50
        # (the oracle walks every new token: keep its rows short)
        c["new"] = [2**31 - 1, 3, 2, 2, 1]
    want = _plan_run(c, T=T)
    assert want["flags"] == 16


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("layout", ["head", "position", "interleaved"])
@pytest.mark.parametrize("D,H,dtype,page", [(128, 2, "bf16", 64), (64, 3, "fp16", 16), (128, 1, "fp16", 128), (64, 8, "bf16", 32)])
def test_append(layout, D, H, dtype, page):
    """Every element of both caches: the rows in their slots, all else as it was.  Some rows have no
    slot, some lie behind the last sequence with slots of anything."""
    for seqs, pad in (([(0, 1)], 0), ([(3, 70), (0, 0), (40, 1), (200, 129)], 9)):
        b = Batch(seqs, Hq=H, Hkv=H, D=D, dtype=dtype, page=page, layout=layout, fused=True, pad=pad, seed=D + H)
        x = b.upload()
        slots = np.full(b.T, 123456789, np.int32)
        slots[:b.rows] = np.random.default_rng(1).permutation(b.P * page)[:b.rows]
        slots[1:b.rows:7] = -1
        moe.gqa_paged_append(b.dims, x["k"], x["v"], dev(slots), x["q_start"], x["kc"], x["vc"], x["ws"])
        assert moe.read_error_flags(x["ws"]) == 0
        kc, vc, _ = P.append(b.k, b.v, slots, b.rows, b.kc, b.vc)
        assert np.array_equal(host(x["kc"]), kc) and np.array_equal(host(x["vc"]), vc)


def test_append_out_of_range():
    b = Batch([(3, 40)], seed=2)
    x = b.upload()
    for bad in (-2, b.P * b.page, 2**31 - 1, -2**31):
        slots = np.arange(40, dtype=np.int32)
        slots[7] = bad
        before = host(x["kc"])
        moe.gqa_paged_append(b.dims, x["k"], x["v"], dev(slots), x["q_start"], x["kc"], x["vc"], x["ws"])
        assert moe.read_error_flags(x["ws"]) == 16
        assert np.array_equal(host(x["kc"]), P.append(b.k, b.v, slots, 40, before, before)[0])


# ---------------------------------------------------------------- the three together
def _serve(page, window, sinks, dtype, graph):
    """Five steps of a served batch whose sequences grow at different paces, two layers, the free list
    counted down in place; every row against the oracle over the sequence's whole history."""
    r = np.random.default_rng(page + window)
    steps = [[40, 0, 7, 129], [1, 65, 1, 1], [1, 1, 0, 30], [16, 1, 1, 1], [1, 1, 1, 1]]
    B, Hq, H, D, T, num, M = 4, 8, 2, 64, 180, 60, 20
    d = moe.gqa_paged_dims(Hq, H, D, page, num, M, B, T, window=window, sinks=sinks, dtype=dtype)
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx, new = torch.zeros(B, **i32), torch.zeros(B, **i32)
    free, n_free, table = dev(r.permutation(num)), torch.full((1,), num, **i32), torch.full((B, M), -1, **i32)
    q_start, kv_len = torch.zeros(B + 1, **i32), torch.zeros(B, **i32)
    positions, slots = torch.zeros(T, **i32), torch.zeros(T, **i32)
    half = dict(dtype=TORCH[dtype], device="cuda")
    caches = [[torch.full((num, H, page, D), float("nan"), **half) for _ in range(2)] for _ in range(2)]
    q, k, v, o = ([torch.zeros((T, h, D), **half) for _ in range(2)] for h in (Hq, H, H, Hq))
    ws = moe.alloc_gqa_paged_workspace(d)

    def step():
        moe.gqa_paged_plan(d, ctx, new, free, n_free, table, q_start, kv_len, positions, slots, n_free, ws)
        for l in range(2):
            moe.gqa_paged_append(d, k[l], v[l], slots, q_start, *caches[l], ws)
            moe.gqa_paged_attention(d, q[l], *caches[l], table, q_start, kv_len, o[l], ws)

    g = None
    if graph:
        step()                       # nothing new: no page taken, no row written
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    history = [[[np.zeros((0, H, D), np.uint16)] * 2 for _ in range(B)] for _ in range(2)]
    for i, lens in enumerate(steps):
        rows = sum(lens)
        new.copy_(dev(np.array(lens)))
        fresh = [[bits(r.standard_normal((T, h, D)), dtype) for h in (Hq, H, H)] for _ in range(2)]
        for l in range(2):
            for t, x in zip((q[l], k[l], v[l]), fresh[l]):
                t.copy_(dev(x, dtype))
            o[l].fill_(7.0)
        g.replay() if graph else step()
        assert moe.read_error_flags(ws) == 0
        at = np.cumsum([0] + lens)
        assert q_start.tolist() == at.tolist()
        assert int(n_free[0]) == num - sum(-(-int(x) // page) for x in kv_len.tolist())
        for l in range(2):
            got = P.to_f64(host(o[l]), dtype)
            assert (got[rows:] == 7.0).all()
            for b in range(B):
                kk, vv = history[l][b] = [np.concatenate([h, x[at[b]:at[b + 1]]]) for h, x in
                                          zip(history[l][b], fresh[l][1:])]
                L = len(kk)
                if L == 0 or lens[b] == 0:
                    continue
                # the history as one page of L positions
                ref, mag, smax = P.attention(fresh[l][0][at[b]:at[b + 1]], kk.transpose(1, 0, 2)[None],
                                             vv.transpose(1, 0, 2)[None], np.array([[0]]), [0, lens[b]], [L], window, sinks,
                                             dtype)
                u = U[dtype]
                tol = u * np.abs(ref) + mag * (u + 2.0 ** -19 + 2 * smax[..., None] * (D // 16 + 2) * 2.0 ** -23)
                if dtype == "fp16":
                    tol = tol + 2.0 ** -25 * (1 + L * 6.0)
                assert (np.abs(got[at[b]:at[b + 1]] - ref) <= tol).all(), (i, l, b)
        ctx.copy_(kv_len)
    return [host(x) for x in o]


@pytest.mark.parametrize("page,window,sinks,dtype", [(16, 0, 0, "bf16"), (32, 50, 4, "fp16"), (128, 0, 0, "fp16"), (64, 20, 0, "bf16")])
def test_serving_steps(page, window, sinks, dtype):
    eager = _serve(page, window, sinks, dtype, graph=False)
    replayed = _serve(page, window, sinks, dtype, graph=True)      # the same step captured once and replayed
    for a, b in zip(eager, replayed):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
@pytest.mark.parametrize("rows", [(64, 96), (96, 128), (64, 128)], ids=["first", "second", "both"])
def test_unseen_values_of_one_tile_beside_a_clean_one(rows, dtype, D):
    """Non-finite values that no row sees, in the leading tile only and there in one of the halves that the chunk form
    searches side by side, before a masked window tile without any: one half takes much longer than the other, tile after
    tile.  The results are those over a finite cache, bit by bit, in every one of many repeats."""
    b = Batch([(c, 40) for c in (700, 1000, 1357, 2000, 431, 900, 1100, 1600)], Hq=16, Hkv=4, D=D, page=128, window=300, sinks=64,
              dtype=dtype, seed=30)
    live = np.zeros((b.P, 1, b.page, 1), bool)
    for s, L in enumerate(b.kv_len):
        for p in range(L):
            page, at = _slot(b, s, p)
            live[page, 0, at] = True
    b.kc, b.vc = np.where(live, b.kc, 0).astype(np.uint16), np.where(live, b.vc, 0).astype(np.uint16)
    clean, flags = b.run()
    assert flags == 0
    b.check(clean)
    for s, (c, _) in enumerate(b.seqs):
        assert 64 <= rows[0] < rows[1] <= c + 1 - 300   # behind the leading positions, before every row's window
        b.kc[b.table[s, 0], :, rows[0]:rows[1]] = b.vc[b.table[s, 0], :, rows[0]:rows[1]] = NAN[dtype]
    o, flags = b.run()
    assert flags == 0 and np.array_equal(o, clean)
    for i in range(100):
        b.dev["o"].fill_(7.0)
        b.attend()
        assert np.array_equal(P.to_f64(host(b.dev["o"]), dtype), clean), i
    assert moe.read_error_flags(b.dev["ws"]) == 0


def _serve_packed(packed, graph):
    """Four steps of three sequences, three layers; the int32 arrays one after the other in one buffer (packed), each 4-byte
    aligned only, or each in its own.  Returns every step's tables and outputs."""
    B, Hq, H, D, page, T, num, M = 3, 8, 2, 64, 16, 90, 40, 9
    steps = [[40, 1, 33], [1, 17, 1], [1, 1, 1], [0, 66, 1]]
    r = np.random.default_rng(31)
    sizes = dict(ctx=B, q_start=B + 1, new=B, kv_len=B, n_free=1, free=num, slots=T, table=B * M, positions=T)
    pool = torch.zeros(1 + sum(sizes.values()), dtype=torch.int32, device="cuda")
    at, x = 1, {}
    for name, n in sizes.items():
        x[name] = pool[at:at + n] if packed else torch.zeros(n, dtype=torch.int32, device="cuda")
        at += n
    x["table"].fill_(-1)
    x["free"].copy_(dev(r.permutation(num)))
    x["n_free"].fill_(num)
    d = moe.gqa_paged_dims(Hq, H, D, page, num, M, B, T)
    ws = moe.alloc_gqa_paged_workspace(d)
    q, k, v = (torch.zeros((3, T, h, D), dtype=torch.bfloat16, device="cuda") for h in (Hq, H, H))
    o = torch.full_like(q, 7.0)
    kc, vc = (torch.full((3, num, H, page, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step():
        moe.gqa_paged_plan(d, x["ctx"], x["new"], x["free"], x["n_free"], x["table"], x["q_start"], x["kv_len"], x["positions"],
                           x["slots"], x["n_free"], ws)
        for l in range(3):
            moe.gqa_paged_append(d, k[l], v[l], x["slots"], x["q_start"], kc[l], vc[l], ws)
            moe.gqa_paged_attention(d, q[l], kc[l], vc[l], x["table"], x["q_start"], x["kv_len"], o[l], ws)

    if graph:
        step()                       # nothing new: no page taken, no row written
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    seen = []
    for lens in steps:
        x["new"].copy_(dev(np.array(lens)))
        for t in (q, k, v):
            t.copy_(torch.stack([dev(bits(r.standard_normal(t.shape[1:]), "bf16"), "bf16") for _ in range(3)]))
        o.fill_(7.0)
        g.replay() if graph else step()
        assert moe.read_error_flags(ws) == 0
        seen.append([t.cpu().numpy().copy() for t in x.values()] + [host(o[l]) for l in range(3)])
        for l in range(3):
            ref, mag, smax = P.attention(host(q[l]), host(kc[l]), host(vc[l]), x["table"].view(B, M).cpu().numpy(),
                                         x["q_start"].cpu().numpy(), x["kv_len"].cpu().numpy())
            tol = 2.0 ** -8 * np.abs(ref) + mag * (2.0 ** -8 + 2.0 ** -19 + 2 * smax[..., None] * (D // 16 + 2) * 2.0 ** -23)
            rows = sum(lens)
            got = P.to_f64(host(o[l]), "bf16")
            assert (np.abs(got - ref)[:rows] <= tol[:rows]).all() and (got[rows:] == 7.0).all()
        x["ctx"].copy_(x["kv_len"])
    return seen


def test_serving_steps_with_every_table_in_one_buffer():
    """A table that one call writes shares its memory sectors with those that calls before it have read: the same tables and
    outputs as with buffers of their own, eager and captured."""
    want = _serve_packed(False, False)
    for graph in (False, True):
        for a, b in zip(_serve_packed(True, graph), want):
            for x, y in zip(a, b):
                assert np.array_equal(x, y)


# ---------------------------------------------------------------- scores of any size
def _far_scores(dtype, scale, seqs, D=128, Hq=4, Hkv=2, window=0):
    """Every score is one exact product of two 16-bit values, scale^2 times 1, 0.5, -0.5 or -1 (its sign and size by
    position), so that the softmax is over equal scores and no rounding of a score can move it."""
    b = Batch(seqs, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, seed=32, window=window)
    size = bits(np.array([scale]), dtype)[0]
    b.q[:] = 0
    b.q[:, :, 3] = size
    levels = bits(scale * np.array(LEVELS[window % 3]), dtype)
    for s, L in enumerate(b.kv_len):
        for i in range(-(-int(L) // b.page)):
            p = i * b.page + np.arange(b.page)
            b.kc[b.table[s, i]] = 0
            b.kc[b.table[s, i], :, :, 3] = levels[p * 7 // 3 % len(levels)]
    return b


LEVELS = [(-1.0,), (-0.5, -1.0), (1.0, 0.5, -1.0)]


def _check_far(b, label):
    """No error of a score (they are exact, and equal where they count): the rounding of the output, of the numerators, and a
    few dozen steps of 2^-24."""
    o, flags = b.run()
    assert flags == 0, flags
    ref, mag, _ = b.oracle()
    u, single = U[b.dtype], b.max_new == 1
    tol = u * np.abs(ref) + mag * ((2.0 ** -17 if single else u) + 2.0 ** -19)
    if b.dtype == "fp16":
        tol = tol + 2.0 ** -25 + int(b.kv_len.max()) * 6.0 * (2.0 ** -40 if single else 2.0 ** -34)
    ratio = (np.abs(o - ref) / tol).max()
    print(f"{label}: max |o - ref| / bar = {ratio:.3f}")
    assert ratio <= 1.0


# q . k / sqrt(D) from 2^20 to the type's end, where the rounding of a score in units of its own size is more than the
# range of the softmax's numerators
FAR = [("bf16", 2.0 ** 12), ("bf16", 2.0 ** 17), ("bf16", 3e4), ("bf16", 1e9), ("bf16", 1.3e16), ("bf16", 7e18),
       ("fp16", 2.0 ** 12), ("fp16", 2.0 ** 13), ("fp16", 2.0 ** 14), ("fp16", 5e4), ("fp16", 65504.0)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype,scale", FAR)
def test_chunks_of_far_scores(dtype, scale, D):
    for window in (300, 301, 302):
        _check_far(_far_scores(dtype, scale, [(0, 1), (0, 5), (300, 30), (700, 3)], D=D, window=window), f"{dtype} {scale} {window}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new,ctx", [(1, 300), (1, 20000), (20, 300), (3, 20000)])
def test_far_scores_close_together(new, ctx, dtype):
    """Scores of 2^20 less a whole number that falls along the cache: the maximum moves again and again, and the weights
    reach over many positions.  (The bar is the usual one: an ulp of a score is what limits it.)"""
    b = Batch([(ctx, new), (40, new), (0, new)], Hq=4, Hkv=2, dtype=dtype, seed=36)
    b.q[:] = 0
    b.q[:, :, 0], b.q[:, :, 70] = bits(np.array([1024.0]), dtype)[0], bits(np.array([1.0]), dtype)[0]
    for s, L in enumerate(b.kv_len):
        for i in range(-(-int(L) // b.page)):
            page = b.table[s, i]
            p = i * b.page + np.arange(b.page)
            b.kc[page] = 0
            b.kc[page, :, :, 0] = bits(np.array([1024.0]), dtype)[0]
            b.kc[page, :, :, 70] = bits(np.maximum(p * 256.0 // int(L) - 256.0, -256.0), dtype)
    _ok(b, f"{dtype} {new} new behind {ctx}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 3])
@pytest.mark.parametrize("scale", [1e9, 1.3e16, 7e18])
def test_far_scores_of_split_rows(scale, new, D):
    """A long sequence cut over many SMs, and short ones; all scores far below zero, and mixed ones."""
    for window in (0, 30001, 30002):
        b = _far_scores("bf16", scale, [(20000, new), (0, new), (60, new)], D=D, Hq=2, Hkv=1, window=window)
        _check_far(b, f"{scale} {new} {window}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype,scale", FAR)
def test_single_tokens_of_far_scores(dtype, scale, D):
    for window in (300, 301, 302):
        _check_far(_far_scores(dtype, scale, [(0, 1), (5, 1), (300, 1), (7000, 1)], D=D, window=window), f"{dtype} {scale} {window}")


# ---------------------------------------------------------------- windows whose items are cut
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("seqs,window,sinks,Hq,Hkv,D,page", [
    ([(20000, 9)], 6000, 0, 6, 2, 128, 64), ([(20000, 9)], 6000, 4, 6, 2, 64, 16), ([(23000, 3)], 6000, 300, 5, 1, 128, 128),
    ([(9000, 40), (30, 2), (15000, 60)], 3000, 130, 3, 1, 64, 32), ([(3000, 1000)], 1024, 4, 12, 4, 128, 64),
    ([(1500, 700), (2100, 300)], 1024, 300, 12, 4, 64, 16), ([(20000, 8)], 17000, 5, 8, 1, 128, 64)])
def test_window_chunks_cut_over_many_sms(seqs, window, sinks, Hq, Hkv, D, page, dtype):
    """Items with a gap between the leading positions and the window, cut into two or three parts (the chunks of hundreds) and
    into 23 to 131: the gap inside a part and between two.  Pages in the gap are gone from the table.  At most some 80 rows
    are checked, spread over the sequences."""
    b = Batch(seqs, Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype, window=window, sinks=sinks, seed=33)
    for s, (c, _) in enumerate(seqs):
        b.table[s, -(-sinks // page):max(c - window + 1, 0) // page] = 1 << 29
    o, flags = b.run()
    assert flags == 0
    table, rows = np.where(b.table >= b.P, 0, b.table), np.arange(0, b.rows, max(1, b.rows // 80))
    ref = [np.zeros(b.q.shape), np.zeros(b.q.shape), np.zeros(b.q.shape[:2])]
    for t in rows:
        s = int(np.searchsorted(b.q_start, t, "right")) - 1
        p = int(b.kv_len[s] - (b.q_start[s + 1] - t))
        one = P.attention(b.q[t:t + 1], b.kc, b.vc, table[s:s + 1], [0, 1], [p + 1], window, sinks, dtype)
        for x, y in zip(ref, one):
            x[t] = y[0]
    b.check(o, ref, rows, label=f"{dtype} window {window} sinks {sinks}")


@pytest.mark.parametrize("value", [0x7F80, 0x7FC0], ids=["inf", "nan"])
@pytest.mark.parametrize("D", [64, 128])
def test_non_finite_values_in_the_last_part_of_a_cut_item(D, value):
    """A value of one of the chunk's own positions, in the masked tiles that end an item cut over many SMs, and one at the
    window's edge that only the first rows see."""
    n, window = 30, 6000
    b = Batch([(20000, n)], Hq=6, Hkv=2, D=D, page=64, window=window, sinks=4, seed=34)
    clean = b.oracle()
    own, edge = _slot(b, 0, 20000 + 12), _slot(b, 0, 20000 - window + 1 + 7)
    b.vc[own[0], 1, own[1], 9] = value
    b.vc[edge[0], 0, edge[1], 40] = value
    o, flags = b.run()
    assert flags == moe.ERR_NON_FINITE
    hit = np.zeros(o.shape, bool)
    hit[12:, 3:, 9] = True        # rows from the position on
    hit[:8, :3, 40] = True        # rows whose window still holds it
    assert not np.isfinite(o[hit]).any()
    b.check(np.where(hit, 0.0, o), tuple(np.where(hit, 0.0, x) if x.ndim == 3 else x for x in clean))


# ---------------------------------------------------------------- fp16, to what the contract states
@pytest.mark.parametrize("new", [1, 30])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks,q_scale", [(0, 0, 1.0), (0, 0, 0.01), (500, 4, 1.0), (0, 0, 6.0)])
def test_fp16_numerators_as_stated(new, D, window, sinks, q_scale):
    """The bar above with what fp16 numerators are stated to lose: 2^-40 of the row's largest where single tokens keep the
    rounding's remainder, 2^-34 in chunks (and 2^-25 where the output itself is subnormal)."""
    b = Batch([(0, new), (3, new), (700, new), (2050, new), (5000, new)], Hq=8, D=D, dtype="fp16", window=window, sinks=sinks,
              q_scale=q_scale, page=32, seed=35)
    o, flags = b.run()
    assert flags == 0
    ref, mag, smax = b.oracle()
    vmax = np.abs(np.nan_to_num(P.to_f64(b.vc, "fp16"), nan=0.0)).max()
    tol = U["fp16"] * np.abs(ref) + mag * ((2.0 ** -22 if new == 1 else 2.0 ** -11) + 2.0 ** -19 +
                                          2 * smax[..., None] * (D // 16 + 2) * 2.0 ** -23)
    tol = tol + 2.0 ** -25 + int(b.kv_len.max()) * vmax * (2.0 ** -40 if new == 1 else 2.0 ** -34)
    ratio = (np.abs(o - ref) / tol).max()
    print(f"fp16, {new} new, D {D}: max |o - ref| / bar = {ratio:.3f}")
    assert ratio <= 1.0
