"""Rotary positions on the GPU against the oracle.

Bar per output element, a pair (x, y) and amplitude A, with u = 2^-8 (bf16) or 2^-11 (fp16) half a step of the type:
  u * |ref|                          the one rounding of the output;
  A (|x| + |y|) * (2^-21 + p * w * 2^-50)   the angle: what is left of a turn in fp32 (pi * 2^-24, under 2^-22), sine and
                                     cosine (2^-23), three fp32 roundings; a table entry is w off by 2^-51 of itself;
  fp16: 2^-25                        subnormal outputs.
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


def check(got, x, positions, w, layout, dtype, amplitude=1.0):
    ref = Q.rotary(x, positions, w, layout, amplitude)
    half = len(w)
    a, b = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    tol = U[dtype] * np.abs(ref) + (2.0 ** -25 if dtype == "fp16" else 0.0)
    pair = np.abs(x[..., a]) + np.abs(x[..., b])
    angle = np.abs(np.asarray(positions, float)[:, None] * w.astype(float))[:, None, :]
    for s in (a, b):
        tol[..., s] += abs(amplitude) * pair * (2.0 ** -21 + angle * 2.0 ** -50)
    assert (np.abs(got - ref) <= tol).all(), (np.abs(got - ref) / np.maximum(tol, 1e-30)).max()
    assert np.array_equal(got[..., 2 * half:], x[..., 2 * half:])


def run(T=5, Hq=3, Hkv=1, D=128, rot=128, layout="half", dtype="bf16", positions=None, in_place=False, fused=False, n_rows=None,
        amplitude=1.0, seed=0, scale=1.0, **scaling):
    r = np.random.default_rng(seed)
    positions = r.integers(0, 40000, T) if positions is None else np.asarray(positions)
    q, k = (bits(r.standard_normal((T, h, D)) * scale, dtype) for h in (Hq, Hkv))
    qd, kd = dev(q, dtype), dev(k, dtype)
    if fused:
        both = torch.cat([qd.reshape(T, -1), kd.reshape(T, -1)], 1)
        qd, kd = both[:, :Hq * D].view(T, Hq, D), both[:, Hq * D:].view(T, Hkv, D)
    qo, ko = (qd, kd) if in_place else (torch.full((T, h, D), 7.0, dtype=TORCH[dtype], device="cuda") for h in (Hq, Hkv))
    rd = moe.gqa_rotary_dims(Hq, Hkv, D, rot, T, layout=layout, dtype=dtype, amplitude=amplitude, q_stride=qd.stride(0),
                             k_stride=kd.stride(0), q_out_stride=qo.stride(0), k_out_stride=ko.stride(0))
    moe.gqa_rotary(rd, qd, kd, dev(positions), moe.gqa_rotary_table(rot, **scaling), qo, ko,
                   n_rows=None if n_rows is None else dev(np.array([n_rows])))
    n = T if n_rows is None else min(max(n_rows, 0), T)
    w = Q.frequencies(rot, **scaling)
    for x, y in ((q, qo), (k, ko)):
        if x.shape[1]:
            got = P.to_f64(host(y), dtype)
            check(got[:n], P.to_f64(x, dtype)[:n], positions[:n], w, layout, dtype, amplitude)
            want = P.to_f64(x, dtype)[n:] if in_place else 7.0
            assert (got[n:] == want).all()
    return qo, ko


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 96), (128, 24), (128, 2), (64, 64), (64, 30), (256, 256), (256, 64), (80, 80),
                                   (80, 52), (8, 8), (8, 2), (96, 4)])
def test_heads_and_parts(D, rot, layout, dtype):
    run(D=D, rot=rot, layout=layout, dtype=dtype, seed=rot)


@pytest.mark.parametrize("T", [1, 2, 607, 608, 609, 613, 2500])
def test_tokens(T):
    run(T=T, Hq=4, Hkv=2, rot=64, seed=T)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("in_place,fused", [(True, False), (True, True), (False, True)])
def test_in_place_and_fused(in_place, fused, layout):
    run(T=9, D=64, rot=48, in_place=in_place, fused=fused, layout=layout, dtype="fp16")


@pytest.mark.parametrize("Hq,Hkv", [(0, 3), (3, 0), (64, 8), (1, 1)])
def test_head_counts(Hq, Hkv):
    run(T=7, Hq=Hq, Hkv=Hkv)


@pytest.mark.parametrize("n_rows", [0, 1, 6, 20, 21, 500, -3])
def test_rows_in_use(n_rows):
    run(T=20, n_rows=n_rows)
    run(T=20, n_rows=n_rows, in_place=True)


def test_positions_far_and_negative():
    run(T=8, positions=[0, 1, -1, -40000, 2**31 - 1, -2**31, 10**6, 123456789])


@pytest.mark.parametrize("scaling", [dict(scaling="linear", factor=8.0), dict(scaling="base", factor=3.5, base=500000.0),
                                     dict(scaling="by_parts", factor=16.0, original=8192, base=1e6),
                                     dict(scaling="by_parts", factor=4.0, original=4096, low=0.0, high=4.0), dict(base=1.0)])
def test_scalings(scaling):
    run(T=6, positions=[0, 5, 4000, 33000, 131071, 1 << 20], amplitude=1.2772588722239781, **scaling)


def test_not_finite_stays_in_its_pair():
    T, D = 3, 64
    x = bits(np.random.default_rng(1).standard_normal((T, 1, D)), "bf16")
    x[1, 0, 5] = 0x7F80
    y = torch.zeros(T, 1, D, dtype=torch.bfloat16, device="cuda")
    rd = moe.gqa_rotary_dims(1, 0, D, D, T)
    moe.gqa_rotary(rd, dev(x, "bf16"), None, dev(np.array([1, 2, 3])), moe.gqa_rotary_table(D), y, None)
    bad = ~torch.isfinite(y).cpu().numpy()
    assert {tuple(i) for i in np.argwhere(bad)} == {(1, 0, 5), (1, 0, 5 + D // 2)}


def test_distances_alone_count():
    """Scores of turned queries and keys are those of any other positions at the same distance."""
    torch.manual_seed(0)
    base = torch.randn(1, 1, 128, device="cuda").bfloat16()
    T, n = 64, 1000003
    rd = moe.gqa_rotary_dims(1, 1, 128, 128, T)
    table = moe.gqa_rotary_table(128)
    x = base.expand(T, 1, 128).contiguous()
    out, size = [], []
    for shift in (0, n):
        qo, ko = torch.empty_like(x), torch.empty_like(x)
        moe.gqa_rotary(rd, x, x, torch.arange(shift, shift + T, dtype=torch.int32, device="cuda"), table, qo, ko)
        out.append(qo[:, 0].double() @ ko[:, 0].double().T)
        size.append(qo[:, 0].double().abs() @ ko[:, 0].double().abs().T)
    # each product has two factors, off by at most 2^-8 of themselves (and by 2^-20 from their angles)
    assert ((out[0] - out[1]).abs() <= 2.02 * 2.0 ** -8 * (size[0] + size[1])).all()


def test_streams_and_capture():
    """On a side stream, and captured and replayed with other positions and rows in the same buffers."""
    T = 33
    x = torch.randn(T, 4, 128, device="cuda").bfloat16()
    pos, n = torch.arange(T, dtype=torch.int32, device="cuda"), torch.tensor([T], dtype=torch.int32, device="cuda")
    rd, table = moe.gqa_rotary_dims(4, 0, 128, 128, T), moe.gqa_rotary_table(128)
    y = torch.zeros_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    moe.gqa_rotary(rd, x, None, pos, table, y, None, n_rows=n, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    want = y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.gqa_rotary(rd, x, None, pos, table, y, None, n_rows=n)
    y.zero_()
    g.replay()
    assert torch.equal(y, want)
    pos += 5
    n.fill_(7)
    y.zero_()
    g.replay()
    z = torch.zeros_like(x)
    moe.gqa_rotary(rd, x, None, pos, table, z, None, n_rows=n)
    assert torch.equal(y, z) and not torch.equal(y[:7], want[:7]) and (y[7:] == 0).all()
