"""The paged cache held in 8 bits on the GPU against the oracle: the append and the read exactly, attention within a bar
that follows from its arithmetic.

Bar per output element of the attention, with u = 2^-8 (bf16) or 2^-11 (fp16), half a step of the type:
  u * |ref|                      the one rounding of the output;
  u_p * mag                      rounding of the softmax numerators (fp16 in both types) before the product with V: 2^-11 in
                                 the chunk form; 2^-17 in the single-token form, which keeps the remainders;
  2 * smax * (D/16 + 4) * 2^-23 * mag   the scores: D/16 tensor-core steps and four fp32 roundings (products with a
                                 block's scale), each within 2^-23 (an accumulator that truncates) of sum_i |q_i k_i| /
                                 sqrt(D) <= smax, moving a numerator by that fraction (the factor 2 also covers its
                                 denominator; log2(e) and ln 2 cancel);
  2^-18 * mag                    exp2 (2 ulp), logarithms of scales, the running sums and rescales in fp32, the merge: a
                                 few dozen steps of 2^-24;
  N max|V| * 2^-33 or 2^-39      numerators below fp16's normal range, held to 2^-25 where the row's largest is 2^9 (chunks)
                                 or 2^15 (single tokens), times codes of at most twice max|V| in their scale's units; in
                                 chunks also values and keys held to 2^-25 of the largest scale beside them;
  fp16: 2^-25                    subnormal outputs.
mag is the same attention over |V|, max|V| the largest value in the cache.
"""
import numpy as np
import pytest
import torch

import bit_quantized_expert_gb300 as moe
from oracle import paged8_oracle as Q
from oracle import paged_oracle as P
from test_gpu_paged import TORCH, U, bits, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_quantized_expert_gb300 import build
    build.build()
    moe.load_library()


def dev8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Batch8:
    """Sequences with (cached, new) positions in shuffled pages.  Codes that no sequence wrote are NaN, and so are the scales
    of blocks that none wrote."""

    def __init__(self, seqs, Hq=16, Hkv=2, D=128, page=64, dtype="bf16", layout="head", fused=False, pad=0, window=0,
                 sinks=0, seed=0, q_scale=1.0, max_new=None, extra_pages=3, spread=2):
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
        self.c = [np.full((self.P, Hkv, page, D), 0x7F, np.uint8) for _ in range(2)]
        self.s = [np.full((self.P, Hkv, page // 16), np.nan, np.float32) for _ in range(2)]
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            live = np.arange(need[b] * page).reshape(-1, page) < kv[b]
            some = np.arange(0, need[b] * page, 16).reshape(-1, page // 16) < kv[b]
            for i in range(2):
                x = Q.to_codes(np.clip(r.standard_normal((need[b], Hkv, page, D)) * 110, -448, 448))
                s = 2.0 ** (r.integers(-7 - spread, -6 + spread, (need[b], Hkv, page // 16)))
                self.c[i][self.table[b, :need[b]]] = np.where(live[:, None, :, None], x, np.uint8(0x7F))
                self.s[i][self.table[b, :need[b]]] = np.where(some[:, None], s, np.nan)
        self.q = bits(r.standard_normal((T, Hq, D)) * q_scale, dtype)
        self.k, self.v = (bits(r.standard_normal((T, Hkv, D)) * np.exp(r.standard_normal((T, Hkv, 1))), dtype) for _ in range(2))
        self.q_start = np.cumsum([0] + [n for _, n in seqs]).astype(np.int32)
        self.kv_len = np.array(kv, np.int32)
        self.T, self.rows, self.fused = T, rows, fused
        self.max_new = max([n for _, n in seqs] + [1]) if max_new is None else max_new

    def upload(self):
        d = self.dtype
        kc, vc = (dev8(x) for x in self.c)
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
        self.dev = dict(q=q, k=k, v=v, kc=kc, vc=vc, ks=dev8(self.s[0]), vs=dev8(self.s[1]), o=o, o_wide=o_wide,
                        table=dev(self.table), q_start=dev(self.q_start), kv_len=dev(self.kv_len),
                        ws=moe.alloc_gqa_paged8_workspace(self.dims))
        return self.dev

    def append(self, stream=None):
        x = self.dev
        moe.gqa_paged8_append(self.dims, x["k"], x["v"], x["table"], x["q_start"], x["kv_len"], x["kc"], x["vc"], x["ks"],
                              x["vs"], x["ws"], stream=stream)

    def attend(self, stream=None):
        x = self.dev
        moe.gqa_paged8_attention(self.dims, x["q"], x["kc"], x["vc"], x["ks"], x["vs"], x["table"], x["q_start"], x["kv_len"],
                                 x["o"], x["ws"], stream=stream)

    def flags(self):
        return moe.read_error_flags(self.dev["ws"])

    def out(self):
        return P.to_f64(host(self.dev["o"]), self.dtype)

    def run(self):
        self.upload()
        self.attend()
        return self.out(), self.flags()

    def caches(self):
        """The cache on the GPU: codes and scales."""
        x = self.dev
        return [x[n].contiguous().cpu().numpy() for n in ("kc", "vc")], [x[n].cpu().numpy() for n in ("ks", "vs")]

    def values(self):
        with np.errstate(invalid="ignore"):
            return [Q.values(c, s, self.page) for c, s in zip(self.c, self.s)]

    def oracle(self):
        k, v = self.values()
        return Q.attention(self.q, k, v, self.table, self.q_start, self.kv_len, self.window, self.sinks, self.dtype)

    def check(self, o, ref=None, rows=None, label="", more=0.0):
        ref, mag, smax = self.oracle() if ref is None else ref
        rows = np.arange(self.rows) if rows is None else rows
        u, n = U[self.dtype], int(self.kv_len.max())
        vmax = np.nan_to_num(np.abs(self.values()[1]), nan=0.0, posinf=0.0).max(initial=0.0)
        single = self.max_new == 1
        tol = u * np.abs(ref) + mag * ((2.0 ** -17 if single else 2.0 ** -11) + 2.0 ** -18 +
                                       2 * smax[..., None] * (self.D // 16 + 4) * 2.0 ** -23)
        tol = tol + n * vmax * (2.0 ** -39 if single else 2.0 ** -33) + (2.0 ** -25 if self.dtype == "fp16" else 0.0) + more
        bad = np.isnan(ref[rows])
        assert np.array_equal(np.isnan(o[rows]), bad), label
        ratio = np.where(bad, 0.0, np.abs(o - ref)[rows] / np.maximum(tol[rows], 1e-300)).max() if len(rows) else 0.0
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


# ---------------------------------------------------------------- append
def _appended(b, flags=0):
    b.upload()
    b.append()
    assert b.flags() == flags
    want_c, want_s, want = Q.append(b.k, b.v, b.table, b.q_start, b.kv_len, b.c, b.s, b.dtype)
    assert want == flags
    got_c, got_s = b.caches()
    for x, y in zip(got_c + got_s, want_c + want_s):
        assert np.array_equal(x, y, equal_nan=True)
    return got_c, got_s


RAGGED = [(0, 1), (1, 1), (15, 1), (16, 1), (17, 2), (31, 20), (0, 16), (0, 33), (5, 0), (100, 64), (63, 1), (64, 3), (200, 130)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_ragged(dtype, page):
    _appended(Batch8(RAGGED, page=page, dtype=dtype, pad=3, seed=page))


@pytest.mark.parametrize("layout", ["position", "interleaved"])
@pytest.mark.parametrize("D", [64, 128])
def test_append_strides(layout, D):
    _appended(Batch8(RAGGED, Hq=6, Hkv=3, D=D, layout=layout, fused=True, pad=2, dtype="fp16", page=32, seed=2))


def test_append_many_sequences():
    _appended(Batch8([(i % 37, i % 3) for i in range(1500)], Hq=2, Hkv=1, D=64, page=16, seed=3))


def test_append_long_prompts():
    _appended(Batch8([(0, 5000), (37, 3000)], Hq=4, Hkv=4, seed=4))


def test_append_values_of_every_size():
    """Zeros, subnormal numbers, the ends of the scales' range, what is past it, infinities and NaN."""
    for dtype, wide in (("bf16", [0.0, -0.0, 1e-40, 1e-30, 2.0 ** -60, 448.0 * 2.0 ** -60, 450 * 2.0 ** -60, 1e15, 448.0 * 2.0 ** 60,
                                  450.0 * 2.0 ** 60, 3e38, np.inf, -np.inf, np.nan]),
                        ("fp16", [0.0, 6e-8, 65504.0, -65504.0, np.inf, np.nan, 57344.0, 57376.0])):
        r = np.random.default_rng(7)
        b = Batch8([(5, 40), (3, 9), (0, 1)], Hq=2, Hkv=2, D=64, dtype=dtype, seed=5)
        for x in (b.k, b.v):
            at = r.integers(0, x.size, 3000)
            x.reshape(-1)[at] = bits(r.choice(wide, 3000), dtype)
        _appended(b, flags=8)
        for x in (b.k, b.v):      # whole blocks of zeros
            x[:] = 0
        _, s = _appended(b)


def test_append_bad_scales_pages_and_rows():
    b = Batch8([(5, 3), (20, 20), (3, 1)], Hq=2, Hkv=1, page=16, seed=8)
    b.s[0][b.table[0, 0], 0, 0] = np.inf
    b.s[1][b.table[2, 0], 0, 0] = 0.75
    b.table[1, 2] = b.P
    _appended(b, flags=16)
    b = Batch8([(5, 3), (20, 4), (3, 1)], Hq=2, Hkv=1, page=16, seed=8)
    before = [x.copy() for x in b.c]
    b.upload()
    x = b.dev
    x["q_start"][1] = 100            # past T, then falling
    b.append()
    assert b.flags() == 16
    got, _ = b.caches()
    touched = {int(b.table[2, 0])}
    for g, w in zip(got, before):
        for p in range(b.P):
            assert p in touched or np.array_equal(g[p], w[p])


def test_append_rows_before_position_0_are_skipped():
    b = Batch8([(0, 9)], Hq=2, Hkv=1, page=16, seed=9)
    b.kv_len[0] = 4
    _appended(b)


def test_append_twice_is_append_once():
    b = Batch8(RAGGED, Hq=4, Hkv=2, seed=10)
    c, s = _appended(b)
    b.append()
    for x, y in zip(b.caches(), (c, s)):
        for u, w in zip(x, y):
            assert np.array_equal(u, w, equal_nan=True)


def test_append_at_once_and_token_by_token_agree_where_scales_do():
    """Constant magnitudes: the scale never grows, so both ways give the same codes."""
    r = np.random.default_rng(3)
    one, many = (Batch8([(0, 50)], Hq=2, Hkv=2, D=64, page=16, seed=11) for _ in range(2))
    x = r.uniform(0.5, 1.0, one.k.shape) * r.choice([-1, 1], one.k.shape)
    x[..., 0] = 1.0
    one.k[:], one.v[:] = bits(x, "bf16"), bits(-x, "bf16")
    c, s = _appended(one)
    many.upload()
    for t in range(50):
        dims = moe.gqa_paged_dims(2, 2, 64, 16, many.P, many.M, 1, 1, max_new=1)
        k, v = (dev(y[t:t + 1], "bf16") for y in (one.k, one.v))
        d = many.dev
        moe.gqa_paged8_append(dims, k, v, d["table"], dev(np.array([0, 1])), dev(np.array([t + 1])), d["kc"], d["vc"], d["ks"],
                              d["vs"], d["ws"])
    for x, y in zip(many.caches(), (c, s)):
        for u, w in zip(x, y):
            assert np.array_equal(u, w, equal_nan=True)


# ---------------------------------------------------------------- read
def _read(b, flags=0):
    x = b.upload()
    k, v = (torch.full_like(x["k"], 7.0) for _ in range(2))
    dims = moe.gqa_paged_dims(b.Hq, b.Hkv, b.D, b.page, b.P, b.M, len(b.seqs), b.T, dtype=b.dtype, max_new=b.max_new,
                              k_stride=k.stride(0), v_stride=v.stride(0), cache_strides=x["kc"].stride()[:3])
    moe.gqa_paged8_read(dims, x["kc"], x["vc"], x["ks"], x["vs"], x["table"], x["q_start"], x["kv_len"], k, v, x["ws"])
    assert b.flags() == flags
    return [P.to_f64(host(t), b.dtype) for t in (k, v)]


def _read_ok(b):
    got = _read(b)
    for y, vals in zip(got, b.values()):
        want = np.full(y.shape, 7.0)
        for i, (c, n) in enumerate(b.seqs):
            for h in range(b.Hkv):
                x = Q.gather(vals, b.table[i], c + n, h)[c:] if n else np.zeros((0, b.D))
                x = np.clip(x, -65504, 65504) if b.dtype == "fp16" else x
                want[b.q_start[i]:b.q_start[i + 1], h] = P.to_f64(bits(x, b.dtype), b.dtype)
        assert np.array_equal(y, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page,D", [(16, 128), (32, 64), (64, 128), (128, 64)])
def test_read_ragged(dtype, page, D):
    _read_ok(Batch8(RAGGED, page=page, D=D, dtype=dtype, pad=3, seed=page))


@pytest.mark.parametrize("layout", ["position", "interleaved"])
def test_read_strides(layout):
    _read_ok(Batch8(RAGGED, Hq=6, Hkv=3, layout=layout, dtype="fp16", page=32, seed=2))


def test_read_long():
    _read_ok(Batch8([(0, 9000), (10, 0), (0, 1), (77, 4000)], Hq=2, Hkv=2, seed=3))


@pytest.mark.parametrize("n", [32, 33, 256, 257, 2000])
def test_append_and_read_sequences(n):
    """On either side of the counts from which on sequences are scanned, and CTAs sized, in another way; blocks for several
    turns of every warp at the last one."""
    seqs = [(5 * i % 67, (i % 5) * (20 if i % 97 == 0 else 1)) for i in range(n)]
    _appended(Batch8(seqs, Hq=4, Hkv=4, D=128, page=32, seed=n))
    _read_ok(Batch8(seqs, Hq=4, Hkv=4, D=128, page=32, seed=n))


def test_read_ends_of_the_types():
    """All codes under the largest and the smallest scales; fp16 ends at 65504."""
    for dtype, scales in (("bf16", [2.0 ** -60, 2.0 ** 60, 2.0]), ("fp16", [2.0 ** 8, 2.0 ** -20, 2.0 ** -60, 2.0 ** 7])):
        b = Batch8([(0, 64)], Hq=2, Hkv=1, D=64, page=64, dtype=dtype, seed=1)
        p = b.table[0, 0]
        for i in range(2):
            b.c[i][p, 0] = (np.arange(64 * 64) % 256).reshape(64, 64)
            b.c[i][p, 0][(b.c[i][p, 0] & 0x7F) == 0x7F] = 0
            b.s[i][p, 0] = np.resize(scales, 4)
        got = _read(b)
        for y, vals in zip(got, b.values()):
            x = (b.values()[0][p, 0].astype(np.float32))
            lim = np.clip(x, -65504, 65504) if dtype == "fp16" else x
            assert np.array_equal(y[:, 0], P.to_f64(bits(lim, dtype), dtype))


def test_read_nan_bad_pages_scales_and_rows_before_0():
    b = Batch8([(0, 40), (0, 20)], Hq=2, Hkv=1, page=16, seed=4)
    b.c[0][b.table[0, 0], 0, 3, 5] = 0xFF
    b.table[0, 1] = -5
    b.s[1][b.table[0, 2], 0, 0] = np.nan
    b.kv_len[1] = 13                    # seven rows before position 0
    k, v = _read(b, flags=16)
    assert np.isnan(k[3, 0, 5]) and np.isnan(k).sum() == 1
    assert (k[16:32] == 0).all() and (v[16:32] == 0).all() and (np.abs(v[32:40]) <= 448 * 2.0 ** -60).all()
    assert (k[40:47] == 0).all() and (k[47:] != 0).any()
    want = P.to_f64(bits(Q.gather(b.values()[0], b.table[1], 13, 0), "bf16"), "bf16")
    assert np.array_equal(k[47:, 0], want)


# ---------------------------------------------------------------- attention: single tokens
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_single_tokens_ragged(dtype, page):
    ctx = [0, 1, 14, 15, 16, 30, 31, 32, 33, 62, 63, 64, 65, 127, 128, 200, 511, 1000, 2049]
    _ok(Batch8([(c, 1) for c in ctx], page=page, dtype=dtype, seed=page), f"{dtype} page {page}")


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 8, 128), (6, 2, 128), (5, 1, 64), (32, 4, 128), (7, 7, 64), (14, 2, 64), (1, 1, 128),
                                      (24, 3, 64)])
def test_single_tokens_head_layouts(Hq, Hkv, D):
    _ok(Batch8([(c, 1) for c in (0, 77, 300, 640)], Hq=Hq, Hkv=Hkv, D=D, page=32, seed=Hq), f"{Hq}/{Hkv} D {D}")


@pytest.mark.parametrize("layout", ["position", "interleaved"])
@pytest.mark.parametrize("D", [64, 128])
def test_single_tokens_strides(layout, D):
    _ok(Batch8([(c, 1) for c in (3, 90, 257)], D=D, layout=layout, fused=True, pad=5, dtype="fp16", page=16, seed=9), layout)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 0), (100, 4), (100, 70), (129, 300), (4000, 4)])
def test_single_tokens_window(window, sinks):
    _ok(Batch8([(c, 1) for c in (0, 1, 63, 99, 100, 163, 500, 1500)], window=window, sinks=sinks, page=16, seed=3),
        f"window {window} sinks {sinks}")


def test_single_tokens_idle_sequences_and_padding():
    _ok(Batch8([(70, 0), (5, 1), (0, 0), (130, 1), (64, 0)], max_new=1, pad=3, seed=4))


def test_single_tokens_long_and_short_together():
    _ok(Batch8([(20000, 1)] + [(c, 1) for c in range(0, 90, 3)] + [(9000, 1)], Hq=8, Hkv=2, seed=5))


def test_single_tokens_many_sequences():
    _ok(Batch8([(c % 23, 1) for c in range(1500)], Hq=2, Hkv=1, D=64, page=16, dtype="fp16", seed=6))


@pytest.mark.parametrize("q_scale", [8.0, 0.01])
def test_single_tokens_peaked_and_flat(q_scale):
    _ok(Batch8([(3000, 1), (100, 1)], q_scale=q_scale, seed=7))


# ---------------------------------------------------------------- attention: chunks
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_chunks_ragged(dtype, page):
    seqs = [(0, 2), (0, 1), (0, 17), (5, 33), (127, 1), (128, 2), (100, 64), (300, 31), (0, 130), (513, 5)]
    _ok(Batch8(seqs, Hq=8, Hkv=1, page=page, dtype=dtype, seed=page), f"{dtype} page {page}")


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 4, 128), (6, 2, 128), (5, 1, 64), (16, 4, 64), (3, 3, 64), (14, 2, 128), (1, 1, 128),
                                      (12, 2, 64)])
def test_chunks_head_layouts(Hq, Hkv, D):
    _ok(Batch8([(0, 70), (200, 45), (37, 1)], Hq=Hq, Hkv=Hkv, D=D, page=32, seed=Hq), f"{Hq}/{Hkv} D {D}")


@pytest.mark.parametrize("layout", ["position", "interleaved"])
@pytest.mark.parametrize("D", [64, 128])
def test_chunks_strides(layout, D):
    _ok(Batch8([(3, 40), (90, 3), (140, 20)], Hq=8, D=D, layout=layout, fused=True, pad=5, dtype="fp16", page=16, seed=9), layout)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (100, 4), (100, 200), (128, 0), (300, 130), (4000, 4)])
def test_chunks_window(window, sinks):
    _ok(Batch8([(0, 150), (400, 70), (1000, 9)], Hq=8, Hkv=2, window=window, sinks=sinks, page=16, seed=3),
        f"window {window} sinks {sinks}")


def test_chunks_idle_sequences_and_padding():
    _ok(Batch8([(70, 0), (5, 20), (0, 0), (130, 1), (64, 0)], pad=130, seed=4))


def test_chunk_over_a_long_cache():
    _ok(Batch8([(6000, 9), (0, 3), (3000, 20)], Hq=4, Hkv=2, seed=5))


@pytest.mark.parametrize("seqs,Hq,Hkv,D", [([(20000, 3)], 8, 1, 128), ([(9000, 40)], 4, 2, 64), ([(6000, 33)], 16, 2, 128),
                                           ([(30000, 2), (50, 4), (7000, 17)], 6, 1, 64)])
def test_few_rows_over_long_caches(seqs, Hq, Hkv, D):
    """Items cut into many parts (up to one a SM), of one row tile and of two."""
    _ok(Batch8(seqs, Hq=Hq, Hkv=Hkv, D=D, seed=29))


@pytest.mark.parametrize("q_scale", [8.0, 0.01])
def test_chunks_peaked_and_flat(q_scale):
    _ok(Batch8([(1000, 40), (100, 30)], Hq=8, q_scale=q_scale, seed=7))


# ---------------------------------------------------------------- attention: scales
@pytest.mark.parametrize("new", [1, 25])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_scales_far_apart(new, dtype):
    """Value scales that differ by up to 2^24 from block to block, in rising, falling and mixed order; key scales by 2^8."""
    for order in (np.arange, lambda n: np.arange(n)[::-1], lambda n: np.random.default_rng(1).permutation(n)):
        b = Batch8([(700, new)], Hq=4, Hkv=2, page=64, dtype=dtype, seed=12)
        n = (700 + new + 15) // 16
        for h in range(2):
            for j, x in enumerate(order(n)):
                page, blk = b.table[0, j // 4], j % 4
                b.s[1][page, h, blk] = 2.0 ** float(-16 + 24 * x // n) if dtype == "bf16" else 2.0 ** float(-18 + 24 * x // n)
                b.s[0][page, h, blk] = 2.0 ** float(-12 + 8 * x // n)
        _ok(b, f"new {new}")


@pytest.mark.parametrize("new", [1, 25])
@pytest.mark.parametrize("span", [20, 26, 30, 40, 66])
def test_value_scales_very_far_apart(new, span):
    """One block's values 2^span above the others', at the end, the start or the middle of a cache: what the others lose is
    little beside it (in chunks up to 2^-24 of it: a scale below that of the largest is taken as 0), and nothing where
    its rows are not seen."""
    for at in (0, 20, 43):
        b = Batch8([(700, new)], Hq=4, Hkv=2, page=64, seed=12, spread=0)
        b.s[1][b.table[0, at // 4], :, at % 4] = 2.0 ** (span - 7)
        o, flags = b.run()
        assert flags == 0
        b.check(o, label=f"span {span} at {at}", more=0.0 if new == 1 else 448 * 2.0 ** (span - 7 - 24))
    b = Batch8([(700, new)], Hq=4, Hkv=2, page=64, seed=12, spread=0, window=300, sinks=16)
    b.s[1][b.table[0, 3], :, 1] = 2.0 ** (span - 7)
    o, flags = b.run()
    assert flags == 0
    ref = b.oracle()
    b.s[1][b.table[0, 3], :, 1] = 2.0 ** -7       # (the bar's largest value is one that rows see)
    b.check(o, ref=ref)


@pytest.mark.parametrize("new", [1, 25])
def test_scales_at_the_ends_of_their_range(new):
    """Whole blocks of zeros under the least scale beside common ones, and a cache under the largest."""
    b = Batch8([(300, new)], Hq=4, Hkv=2, page=16, seed=14)
    for i in range(2):
        for j in range(0, 300 // 16, 3):
            b.c[i][b.table[0, j]] = 0
            b.s[i][b.table[0, j]] = 2.0 ** -60
    _ok(b, "zeros")
    b = Batch8([(100, new)], Hq=4, Hkv=2, page=16, seed=15, q_scale=2.0 ** -60)
    b.s[0][:] = np.where(np.isnan(b.s[0]), np.nan, 2.0 ** 56)
    b.s[1][:] = np.where(np.isnan(b.s[1]), np.nan, 2.0 ** 60)
    _ok(b, "large")
    b = Batch8([(100, new)], Hq=4, Hkv=2, page=16, seed=15, q_scale=2.0 ** 50)
    b.s[0][:] = np.where(np.isnan(b.s[0]), np.nan, 2.0 ** -60)
    b.s[1][:] = np.where(np.isnan(b.s[1]), np.nan, 2.0 ** -60)
    _ok(b, "small")


@pytest.mark.parametrize("new", [1, 25])
def test_queries_of_any_size(new):
    """Rows and heads of very different sizes, elements far below their row's largest, rows of zeros."""
    b = Batch8([(200, new), (30, new)], Hq=8, Hkv=2, seed=16)
    r = np.random.default_rng(3)
    x = r.standard_normal(b.q.shape) * 2.0 ** r.integers(-70, 3, b.q.shape[:2])[..., None]
    x *= 2.0 ** -r.integers(0, 30, b.q.shape).astype(float)
    x[0, 1] = 0.0
    b.q[:] = bits(x, "bf16")
    _ok(b)


@pytest.mark.parametrize("new", [1, 20])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_weight_spread_over_tiny_numerators(new, dtype):
    """One position e^18 above all others, which alone have values, so that numerators far below 1 carry the result."""
    b = Batch8([(4000, new)], Hq=1, Hkv=1, dtype=dtype, page=64, seed=17, spread=0)
    b.q[:] = 0
    b.q[..., 0] = bits(np.array([16.0]), dtype)[0]
    for i in range(2):
        b.s[i][:] = np.where(np.isnan(b.s[i]), np.nan, 2.0 ** -5)
    k = np.zeros((b.M * 64, 128))
    k[5, 0] = 18.0 * np.sqrt(128.0) / 16.0
    for j in range(4000 + new):
        b.c[0][b.table[0, j // 64], 0, j % 64] = Q.to_codes(k[j] * 32)
    b.c[1][b.table[0, 0], 0, 5] = 0
    _ok(b)


@pytest.mark.parametrize("new", [1, 30])
def test_scores_that_grow_along_the_cache(new):
    """Every key is a larger multiple of the query than the one before it: the running maximum moves at every tile."""
    b = Batch8([(900, new)], Hq=4, Hkv=1, seed=8, q_scale=0.5, page=64)
    q = P.to_f64(b.q[0, 0], "bf16")
    for blk in range((900 + new + 15) // 16):
        x = np.outer(np.arange(blk * 16 + 1, blk * 16 + 17) / 60.0, q)
        e = Q.exponent(np.abs(x).max())
        page, off = b.table[0, blk // 4], blk % 4 * 16
        live = np.arange(blk * 16, blk * 16 + 16) < 900 + new
        b.c[0][page, 0, off:off + 16] = np.where(live[:, None], Q.to_codes(x / 2.0 ** e), np.uint8(0x7F))
        b.s[0][page, 0, blk % 4] = 2.0 ** e
    b.q[:] = b.q[0, 0]
    _ok(b)


@pytest.mark.parametrize("new", [1, 30])
@pytest.mark.parametrize("size", [2.0 ** 14, 2.0 ** 24, 2.0 ** 40])
def test_scores_of_any_size(new, size):
    """One dim carries the scores, exact multiples of `size`: a row's result is the mean of the values at its largest one."""
    b = Batch8([(300, new)], Hq=2, Hkv=1, D=64, seed=18, page=16, spread=0)
    n = 300 + new
    r = np.random.default_rng(4)
    levels = r.integers(-4, 5, n).astype(float)
    levels[:20] = -levels[20]
    b.q[:] = 0
    b.q[..., 7] = bits(np.array([8.0]), "bf16")[0]
    b.s[0][:] = np.where(np.isnan(b.s[0]), np.nan, size)
    for j in range(n):
        x = np.zeros(64)
        x[7] = levels[j]
        b.c[0][b.table[0, j // 16], 0, j % 16] = Q.to_codes(x)
    ref, mag, _ = b.oracle()
    # the scores are exact up to one rounding of a product by a scale, the same for equal scores
    o, flags = b.run()
    assert flags == 0
    b.check(o, ref=(ref, mag, np.zeros(ref.shape[:2])), label=f"{size}")


# ---------------------------------------------------------------- attention: what rows do not see, and bad tables
def _row_of_nan(b, seq, pos, which, dims=(3,)):
    b.c[which][b.table[seq, pos // b.page], :, pos % b.page, list(dims)] = 0x7F


@pytest.mark.parametrize("new", [1, 40])
def test_nan_where_rows_see_it(new):
    """NaN values and keys: rows that see the position have NaN, the others are not touched."""
    b = Batch8([(300, new), (70, new)], Hq=4, Hkv=2, seed=19, page=32)
    _row_of_nan(b, 0, 100, 1)
    if new > 1:
        _row_of_nan(b, 1, 90, 1, dims=(0, 127))     # seen by the last rows alone
        _row_of_nan(b, 0, 320, 1, dims=(64,))
    o, flags = b.run()
    assert flags == 8
    b.check(o)
    b = Batch8([(300, new), (70, new)], Hq=4, Hkv=2, seed=20, page=32)
    _row_of_nan(b, 1, 70 + new - 1, 0)              # a key that the last row alone sees
    ref, mag, smax = b.oracle()
    ref[b.rows - 1] = np.nan
    o, flags = b.run()
    assert flags == 8 and np.isnan(o[b.rows - 1]).all()
    b.check(o, ref=(ref, mag, smax))


@pytest.mark.parametrize("new", [1, 40])
def test_window_hides_nan_and_bad_tables(new):
    """What a window has passed may be NaN, under any scale, in pages that were freed."""
    b = Batch8([(900, new), (500, new)], Hq=4, Hkv=2, window=100, sinks=5, seed=21, page=16)
    for s, c in ((0, 900), (1, 500)):
        for page_at in range(1, (c - 100) // 16 - 1):
            if page_at % 3 == 0:
                b.table[s, page_at] = -77
            elif page_at % 3 == 1:
                b.c[0][b.table[s, page_at]] = 0x7F
                b.c[1][b.table[s, page_at]] = 0xFF
            for w in range(2):
                if page_at % 3:
                    b.s[w][b.table[s, page_at]] = [np.inf, -1.0][page_at % 2]
        for pos in (5, 7, 15):                      # behind the leading positions, in their page
            _row_of_nan(b, s, pos, 0)
            _row_of_nan(b, s, pos, 1)
    _ok(b)


@pytest.mark.parametrize("new", [1, 9])
def test_rows_that_see_nothing(new):
    b = Batch8([(0, new), (40, new)], Hq=4, Hkv=1, seed=22, max_new=new)
    b.kv_len[0] = new - 1 if new > 1 else 0
    o, flags = b.run()
    assert flags == 0 and (o[0] == 0).all()
    b.check(o)


@pytest.mark.parametrize("new", [1, 9])
def test_bad_pages_lengths_and_scales(new):
    b = Batch8([(200, new), (60, new), (30, new)], Hq=4, Hkv=2, page=16, seed=23)
    b.table[0, 3] = b.P + 5
    b.table[1, 1] = -2
    o, flags = b.run()
    assert flags == 16
    b.check(o)
    b = Batch8([(200, new), (60, new)], Hq=4, Hkv=2, page=16, seed=24)
    b.s[0][b.table[0, 2], :, 0] = np.nan
    b.s[1][b.table[0, 5], :, 0] = 2.0 ** 61
    b.s[1][b.table[1, 1], :, 0] = 0.0
    b.s[1][b.table[0, 7], :, 0] = 0.0123
    o, flags = b.run()
    assert flags == 16
    for w, p in ((0, b.table[0, 2]), (1, b.table[0, 5]), (1, b.table[1, 1]), (1, b.table[0, 7])):
        b.s[w][p, :, 0] = 2.0 ** -60
    b.check(o)
    b = Batch8([(200, new), (60, new)], Hq=4, Hkv=2, page=16, seed=25)
    b.upload()
    b.dev["kv_len"][0] = 1 << 29
    b.dev["q_start"][1] = -4
    b.attend()
    assert b.flags() & 16


def test_chunk_rows_past_max_new():
    b = Batch8([(20, 30), (5, 12)], Hq=4, Hkv=2, seed=26, max_new=20)
    o, flags = b.run()
    assert flags == 16
    b.check(o, rows=np.r_[0:20, 30:42])
    assert (o[20:30] == 7.0).all()


# ---------------------------------------------------------------- attention: repeats, streams, graphs, offsets
@pytest.mark.parametrize("new", [1, 50])
def test_repeats_bit_by_bit_and_on_two_streams(new):
    a, b = (Batch8([(3000, new), (100, new), (40, new)], seed=s) for s in (27, 28))
    for x in (a, b):
        x.upload()
        x.attend()
    first = [x.dev["o"].clone() for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x in zip(streams, (a, b)):
            x.attend(stream=s)
    torch.cuda.synchronize()
    for x, y in zip((a, b), first):
        assert torch.equal(x.dev["o"], y) and x.flags() == 0


def test_graphs_that_share_a_workspace():
    """Single tokens and chunks, each in a graph of its own, one workspace: replayed in turn on one stream."""
    batches = [Batch8([(3000, 1), (70, 1)], seed=33), Batch8([(2000, 90), (500, 30)], seed=34)]
    for x in batches:
        x.upload()
    ws = max((x.dev["ws"] for x in batches), key=torch.numel)
    graphs, first = [], []
    for x in batches:
        x.dev["ws"] = ws
        x.attend()
        torch.cuda.synchronize()
        first.append(x.dev["o"].clone())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            x.attend()
    for _ in range(4):
        for x in batches:
            x.dev["o"].zero_()
        for g in graphs:
            g.replay()
        for x, y in zip(batches, first):
            assert torch.equal(x.dev["o"], y)
    assert all(x.flags() == 0 for x in batches)


@pytest.mark.parametrize("new", [1, 20])
def test_caches_past_32_bit_offsets(new):
    """A cache whose pages lie more than 2^32 bytes apart."""
    b = Batch8([(150, new)], Hq=2, Hkv=1, D=64, page=16, seed=30)
    b.upload()
    x = b.dev
    stride = 1 << 30
    big = torch.zeros((b.P - 1) * stride + 16 * 64, dtype=torch.uint8, device="cuda")
    for n in ("kc", "vc"):
        view = big.as_strided((b.P, 1, 16, 64), (stride, 1024, 64, 1), 0 if n == "kc" else 0)
        view.copy_(x["kc"])
        x[n] = view
    b.c[1], b.s[1] = b.c[0], b.s[0]
    x["vs"] = x["ks"]
    b.dims = moe.gqa_paged_dims(2, 1, 64, 16, b.P, b.M, 1, b.T, max_new=new, cache_strides=x["kc"].stride()[:3])
    b.attend()
    assert b.flags() == 0
    b.check(b.out())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_serving_steps(dtype):
    """Prompts, then tokens, all through the public calls as they would be used: plan, rotary positions, append, attention,
    and the cache read back; then the token step captured and replayed as the lengths grow."""
    B, Hq, Hkv, D, S, M, pages = 3, 8, 2, 64, 32, 8, 20
    i32 = dict(dtype=torch.int32, device="cuda")
    r = np.random.default_rng(31)
    free, n_free = dev(r.permutation(pages)), torch.tensor([pages], **i32)
    table, ctx = torch.full((B, M), -1, **i32), torch.zeros(B, **i32)
    kc, vc = (torch.zeros((pages, Hkv, S, D), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, Hkv, S // 16), device="cuda") for _ in range(2))
    turns, w = moe.gqa_rotary_table(48), Q.frequencies(48)
    oc = [np.zeros((pages, Hkv, S, D), np.uint8) for _ in range(2)]
    osc = [np.zeros((pages, Hkv, S // 16), np.float32) for _ in range(2)]

    def step(new, buffers=None, graph=None):
        T = B * max(new)
        if buffers is None:
            dims = moe.gqa_paged_dims(Hq, Hkv, D, S, pages, M, B, T, max_new=max(new), dtype=dtype)
            x = {n: torch.empty((T, h, D), dtype=TORCH[dtype], device="cuda") for n, h in
                 (("q", Hq), ("k", Hkv), ("v", Hkv), ("o", Hq))}
            x.update(dims=dims, rd=moe.gqa_rotary_dims(Hq, Hkv, D, 48, T, dtype=dtype), n=torch.tensor(new, **i32),
                     q_start=torch.zeros(B + 1, **i32), kv_len=torch.zeros(B, **i32), pos=torch.zeros(T, **i32),
                     slots=torch.zeros(T, **i32), ws=moe.alloc_gqa_paged8_workspace(dims))
        else:
            x = buffers
        h = {n: bits(r.standard_normal(x[n].shape), dtype) for n in "qkv"}
        for n in "qkv":
            x[n].copy_(dev(h[n], dtype))

        def calls():
            moe.gqa_paged_plan(x["dims"], ctx, x["n"], free, n_free, table, x["q_start"], x["kv_len"], x["pos"], x["slots"],
                               n_free, x["ws"])
            moe.gqa_rotary(x["rd"], x["q"], x["k"], x["pos"], turns, x["q"], x["k"], n_rows=x["q_start"][B:])
            moe.gqa_paged8_append(x["dims"], x["k"], x["v"], table, x["q_start"], x["kv_len"], kc, vc, ks, vs, x["ws"])
            moe.gqa_paged8_attention(x["dims"], x["q"], kc, vc, ks, vs, table, x["q_start"], x["kv_len"], x["o"], x["ws"])
            ctx.copy_(x["kv_len"])
        if graph is None:
            calls()
        else:
            graph.replay()
        q_start, kv_len = x["q_start"].cpu().numpy(), x["kv_len"].cpu().numpy()
        rows, tab = int(q_start[-1]), table.cpu().numpy()
        assert moe.read_error_flags(x["ws"]) == 0 and rows == sum(new)
        pos = x["pos"].cpu().numpy()
        qr, kr = host(x["q"]), host(x["k"])
        for got, was in ((qr, h["q"]), (kr, h["k"])):
            want = Q.rotary(P.to_f64(was, dtype)[:rows], pos[:rows], w, "half")
            size = np.abs(P.to_f64(was, dtype)[:rows]).max()
            assert (np.abs(P.to_f64(got, dtype)[:rows] - want) <= U[dtype] * np.abs(want) + 2 * size * 2.0 ** -20).all()
        nonlocal oc, osc
        oc, osc, flags = Q.append(kr, h["v"], tab, q_start, kv_len, oc, osc, dtype)
        assert flags == 0
        for a, b in ((kc, oc[0]), (vc, oc[1])):
            assert np.array_equal(a.view(torch.uint8).cpu().numpy(), b)
        for a, b in ((ks, osc[0]), (vs, osc[1])):
            assert np.array_equal(a.cpu().numpy(), b)
        vals = [Q.values(c, s, S) for c, s in zip(oc, osc)]
        ref, mag, smax = Q.attention(qr, vals[0], vals[1], tab, q_start, kv_len, dtype=dtype)
        o = P.to_f64(host(x["o"]), dtype)[:rows]
        ref, mag, smax = ref[:rows], mag[:rows], smax[:rows]
        bar = U[dtype] * np.abs(ref) + mag * (2.0 ** -11 + 2.0 ** -18 + 2 * smax[..., None] * 8 * 2.0 ** -23) + \
            256 * np.abs(vals[1]).max() * 2.0 ** -33 + 2.0 ** -25
        assert (np.abs(o - ref) <= bar).all()
        k, v = (torch.zeros((int(kv_len.sum()), Hkv, D), dtype=TORCH[dtype], device="cuda") for _ in range(2))
        rdims = moe.gqa_paged_dims(Hq, Hkv, D, S, pages, M, B, len(k), dtype=dtype)
        start = np.concatenate([[0], np.cumsum(kv_len)]).astype(np.int32)
        moe.gqa_paged8_read(rdims, kc, vc, ks, vs, table, dev(start), x["kv_len"], k, v, moe.alloc_gqa_paged8_workspace(rdims))
        for y, val in ((k, vals[0]), (v, vals[1])):
            for b in range(B):
                for g in range(Hkv):
                    want = bits(Q.gather(val, tab[b], int(kv_len[b]), g), dtype)
                    assert np.array_equal(host(y)[start[b]:start[b + 1], g], want)
        return x, calls

    step([40, 3, 64])
    step([1, 20, 0])
    x, calls = step([1, 1, 1])
    saved = ctx.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    assert torch.equal(ctx, saved)
    for _ in range(4):
        step([1, 1, 1], buffers=x, graph=g)
