"""The 8-bit cache's and the rotary positions' oracle against fixed facts."""
import math

import numpy as np
import pytest
import torch

from oracle import paged8_oracle as Q
from oracle import paged_oracle as P


def test_codes_by_hand():
    for code, value in ((0x00, 0.0), (0x01, 2.0 ** -9), (0x07, 7 * 2.0 ** -9), (0x08, 2.0 ** -6), (0x38, 1.0), (0x3C, 1.5),
                        (0x7E, 448.0), (0xFE, -448.0), (0xB8, -1.0)):
        assert Q.VALUES[code] == value
    assert math.isnan(Q.VALUES[0x7F]) and math.isnan(Q.VALUES[0xFF])
    assert np.array_equal(Q.to_f64(np.arange(256)), torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy(),
                          equal_nan=True)


def test_every_code_returns_and_ties_go_to_even():
    c = np.array([x for x in range(256) if x not in (0x7F, 0xFF)], np.uint8)
    assert (Q.to_codes(Q.to_f64(c)) == c).all()
    mags = Q.VALUES[:0x7F]
    mid = (mags[1:] + mags[:-1]) / 2
    got = Q.to_codes(mid)
    assert (got % 2 == 0).all() and (np.abs(got.astype(int) - np.arange(0.5, 0x7E)) == 0.5).all()
    assert Q.to_codes([460.0, math.nan]).tolist() == [0x7E, 0x7F]


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.1, 1), (224.0, -1), (224.1, 0), (0.0, -60), (1.0, -8), (2.0 ** 69, 60),
                                    (1e-30, -60)])
def test_exponents(amax, e):
    assert Q.exponent(amax) == e


def _bits(x):
    return torch.tensor(np.asarray(x, np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)


def test_append_by_hand():
    """Two positions behind three held ones: the scale grows from 1/4 to 1, the held codes are rounded once more, what lies
    behind stays."""
    cache = np.full((1, 1, 16, 1), 0x11, np.uint8)
    held = [1.0, 3.75, 100.0]
    cache[0, 0, :3, 0] = Q.to_codes(np.array(held))
    scale = np.full((1, 1, 1), 0.25, np.float32)
    k = _bits([300.0, -7.0]).reshape(2, 1, 1)
    (kc, _), (ks, _), flags = Q.append(k, k, [[0]], [0, 2], [5], (cache, cache), (scale, scale), "bf16")
    assert flags == 0 and ks[0, 0, 0] == 1.0
    got = Q.to_f64(kc[0, 0, :, 0])
    assert got[:3].tolist() == [0.25, 0.9375, 24.0]   # 100, between 96 and 104, is held as 96 (even), a quarter of which is a code
    assert got[3:5].tolist() == [288.0, -7.0]         # 300 between 288 and 320
    assert (kc[0, 0, 5:, 0] == 0x11).all()


def test_append_leaves_out_what_is_not_finite():
    cache, scale = np.zeros((1, 1, 16, 2), np.uint8), np.ones((1, 1, 1), np.float32)
    k = _bits([[1.0, math.inf], [math.nan, -2.0]]).reshape(2, 1, 2)
    (kc, _), (ks, _), flags = Q.append(k, k, [[0]], [0, 2], [2], (cache, cache), (scale, scale), "bf16")
    assert flags == Q.NON_FINITE and ks[0, 0, 0] == 2.0 ** -7
    assert kc[0, 0, 0, 1] == kc[0, 0, 1, 0] == 0x7F and (Q.to_f64(kc[0, 0, :2]) * 2.0 ** -7)[0, 0] == 1.0


@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 0), (5, 3)])
def test_attention_is_that_of_the_16_bit_oracle(window, sinks):
    """On values that both caches hold exactly."""
    r = np.random.default_rng(1)
    k, v = (r.integers(-8, 9, (3, 2, 16, 8)) / 8.0 for _ in range(2))
    q = _bits(r.standard_normal((9, 4, 8)))
    table, q_start, kv_len = [[2, 0], [1, -1]], [0, 7, 9], [30, 11]
    a = P.attention(q, _bits(k), _bits(v), np.array(table), q_start, kv_len, window, sinks)
    kq, vq = (Q.values(Q.to_codes(x * 4), np.full((3, 2, 1), 0.25), 16) for x in (k, v))
    b = Q.attention(q, kq, vq, table, q_start, kv_len, window, sinks)
    for x, y in zip(a, b):
        assert np.allclose(x, y, rtol=1e-12, atol=1e-14)


def test_rotary_facts():
    w = Q.frequencies(8, base=16.0)
    assert np.allclose(w.astype(float), [1, 0.5, 0.25, 0.125])
    x = np.arange(10.0).reshape(1, 1, 10)
    for layout in ("half", "interleaved"):
        assert np.array_equal(Q.rotary(x, [0], w, layout), x)
        y = Q.rotary(x, [7], w, layout, amplitude=2.0)
        assert np.array_equal(y[..., 8:], x[..., 8:]) and math.isclose((y[..., :8] ** 2).sum(), 4 * (x[..., :8] ** 2).sum())
        assert np.allclose(Q.rotary(Q.rotary(x, [7], w, layout), [-7], w, layout), x)
    y = Q.rotary(x, [1], w, "half")
    assert math.isclose(y[0, 0, 0], 0 * math.cos(1) - 4 * math.sin(1)) and math.isclose(y[0, 0, 4], 4 * math.cos(1))
    y = Q.rotary(x, [1], w, "interleaved")
    assert math.isclose(y[0, 0, 2], 2 * math.cos(0.5) - 3 * math.sin(0.5))


def test_scaled_frequencies():
    w = Q.frequencies(64).astype(float)
    assert np.allclose(Q.frequencies(64, scaling="linear", factor=4.0).astype(float), w / 4)
    b = Q.frequencies(64, scaling="base", factor=4.0).astype(float)
    assert b[0] == 1.0 and math.isclose(b[-1], w[-1] / 4)
    p = Q.frequencies(64, scaling="by_parts", factor=4.0, original=2048).astype(float)
    turns = 2048 * w / (2 * math.pi)
    assert np.allclose(p[turns >= 32], w[turns >= 32]) and np.allclose(p[turns <= 1], w[turns <= 1] / 4)
    assert ((p <= w * (1 + 1e-12)) & (p >= w / 4 * (1 - 1e-12))).all()
