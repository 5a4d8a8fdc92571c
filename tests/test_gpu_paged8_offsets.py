"""The 8-bit paged cache with pages, heads or positions more than 2^32 bytes apart, keys and values in one buffer at offsets
of their own: the append and the read exactly, the attention within its bar."""
import numpy as np
import pytest
import torch

import bit_quantized_expert_gb300 as moe
from oracle import paged8_oracle as Q
from oracle import paged_oracle as P
from test_gpu_paged import bits, host
from test_gpu_paged8 import Batch8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_quantized_expert_gb300 import build
    build.build()
    moe.load_library()


def spread_out(b, strides, v_offset):
    """b's caches as views of one buffer: keys at 0, values at v_offset."""
    x = b.upload()
    last = sum((n - 1) * s for n, s in zip((b.P, b.Hkv, b.page), strides)) + b.D
    big = torch.zeros(last + v_offset, dtype=torch.uint8, device="cuda")
    for n, at in (("kc", 0), ("vc", v_offset)):
        view = big.as_strided((b.P, b.Hkv, b.page, b.D), (*strides, 1), at)
        view.copy_(x[n])
        x[n] = view
    b.dims = moe.gqa_paged_dims(b.Hq, b.Hkv, b.D, b.page, b.P, b.M, len(b.seqs), b.T, max_new=b.max_new, dtype=b.dtype,
                                cache_strides=strides)
    return x


# strides in bytes of pages, heads, positions; where the values lie
FAR = [((1 << 30, 1 << 28, 64), 1 << 29), ((1 << 30, 64, 1 << 26), 1 << 25), ((4096, 5 << 30, 64), 1 << 31)]


@pytest.mark.parametrize("strides,v_offset", FAR)
@pytest.mark.parametrize("new", [1, 20])
def test_append_read_and_attention(strides, v_offset, new):
    b = Batch8([(100, new), (31, new), (0, new)], Hq=4, Hkv=2, D=64, page=16, dtype="fp16", seed=30)
    x = spread_out(b, strides, v_offset)
    b.append()
    assert b.flags() == 0
    b.c, b.s, flags = Q.append(b.k, b.v, b.table, b.q_start, b.kv_len, b.c, b.s, b.dtype)
    assert flags == 0
    codes, scales = b.caches()
    for got, want in zip(codes + scales, b.c + b.s):
        assert np.array_equal(got, want, equal_nan=True)
    k, v = (torch.full_like(x["k"], 7.0) for _ in range(2))
    moe.gqa_paged8_read(b.dims, x["kc"], x["vc"], x["ks"], x["vs"], x["table"], x["q_start"], x["kv_len"], k, v, x["ws"])
    for y, vals in zip((k, v), b.values()):
        for i, (c, n) in enumerate(b.seqs):
            for h in range(b.Hkv):
                want = bits(Q.gather(vals, b.table[i], c + n, h)[c:], b.dtype)
                assert np.array_equal(P.to_f64(host(y)[b.q_start[i]:b.q_start[i + 1], h], b.dtype), P.to_f64(want, b.dtype))
    b.attend()
    assert b.flags() == 0
    b.check(b.out())
