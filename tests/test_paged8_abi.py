"""Host-side refusals of the calls on an 8-bit paged cache and of the rotary positions (include/gqa_paged8.h,
include/gqa_rotary.h): every call below returns from the argument checks before any CUDA work is enqueued, so no GPU is
needed.  And the table of frequencies, which is made on the host."""
import ctypes
import os

import numpy as np
import pytest

import bit_quantized_expert_gb300 as moe
from oracle import paged8_oracle as Q

INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from bit_quantized_expert_gb300 import build
        build.build()
    return moe.load_library()


GOOD = dict(n_heads=16, n_kv_heads=2, head_dim=128, page_size=64, num_pages=100, max_pages=20, n_seqs=4, n_tokens=37)
ORDER = {"append": ("k", "v", "table", "q_start", "kv_len", "kc", "vc", "ks", "vs", "ws"),
         "read": ("kc", "vc", "ks", "vs", "table", "q_start", "kv_len", "k", "v", "ws"),
         "attention": ("q", "kc", "vc", "ks", "vs", "table", "q_start", "kv_len", "o", "ws")}


def _call(lib, name, d, **kw):
    nb = lib.gqa_paged8_workspace_bytes(ctypes.byref(moe.gqa_paged_dims(**GOOD)))
    return getattr(lib, "gqa_paged8_" + name)(ctypes.byref(d), *[kw.get(n, 256) for n in ORDER[name]], kw.get("nb", nb), None)


@pytest.mark.parametrize("name", list(ORDER))
def test_pointers_and_workspace(lib, name):
    d = moe.gqa_paged_dims(**GOOD)
    for p in ORDER[name]:
        assert _call(lib, name, d, **{p: None}) == INVALID, p
        assert _call(lib, name, d, **{p: 258 if p in ("table", "q_start", "kv_len") else 264}) == MISALIGNED, p
    assert _call(lib, name, d, nb=lib.gqa_paged8_workspace_bytes(ctypes.byref(d)) - 1) == WORKSPACE
    assert getattr(lib, "gqa_paged8_" + name)(None, *[256] * 10, 1 << 30, None) == INVALID


@pytest.mark.parametrize("bad,status", [
    (dict(n_heads=0), INVALID), (dict(n_heads=15), INVALID), (dict(page_size=0), INVALID), (dict(window=-1), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(n_heads=18), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED), (dict(n_seqs=4097), UNSUPPORTED), (dict(num_pages=1 << 24), UNSUPPORTED),
    (dict(q_stride=2052), MISALIGNED), (dict(k_stride=248), INVALID),
    (dict(cache_strides=(20480, 10240, 136)), MISALIGNED), (dict(cache_strides=(16392, 8192, 128)), MISALIGNED),
    (dict(cache_strides=(16384, 8192, 64)), INVALID), (dict(cache_strides=(16384, 8064, 128)), INVALID)])
def test_dims_refused(lib, bad, status):
    d = moe.gqa_paged_dims(**{**GOOD, **bad})
    assert lib.gqa_paged8_workspace_bytes(ctypes.byref(d)) == 0
    for name in ORDER:
        assert _call(lib, name, d) == status
        assert _call(lib, name, d, ws=None) == status
    with pytest.raises(moe.MoeError):
        moe.alloc_gqa_paged8_workspace(d)


@pytest.mark.parametrize("extra", [
    {}, dict(page_size=16), dict(page_size=128), dict(head_dim=64), dict(dtype="fp16"), dict(max_new=1), dict(window=100, sinks=4),
    dict(cache_strides=(16384, 128, 256)), dict(cache_strides=(32768, 8192, 128)), dict(cache_strides=(128, 12800, 25600)),
    dict(head_dim=64, cache_strides=(8192, 4096, 64))])
def test_dims_accepted(lib, extra):
    d = moe.gqa_paged_dims(**{**GOOD, **extra})
    n = lib.gqa_paged8_workspace_bytes(ctypes.byref(d))
    assert n >= 256 and n >= lib.gqa_paged_workspace_bytes(ctypes.byref(d))     # it serves the plan as well


def test_one_address_for_two_outputs(lib):
    """What a call writes for keys and for values lies apart; where it only reads them, one cache may be both."""
    d = moe.gqa_paged_dims(**GOOD)
    apart = dict(kc=1 << 20, vc=1 << 21, ks=1 << 22, vs=1 << 23)
    assert _call(lib, "append", d, **{**apart, "vc": apart["kc"]}) == INVALID
    assert _call(lib, "append", d, **{**apart, "vs": apart["ks"]}) == INVALID
    assert _call(lib, "read", d, **apart, k=1 << 24, v=1 << 24) == INVALID


@pytest.mark.parametrize("name", list(ORDER))
def test_nothing_to_do(lib, name):
    none = {p: None for p in ORDER[name]}
    for key in ("n_seqs", "n_tokens"):
        assert _call(lib, name, moe.gqa_paged_dims(**{**GOOD, key: 0}), **none) == 0


def test_binding_refuses_other_caches_and_scales():
    import torch
    moe._load_paged_types()
    host = -1   # what a host tensor gives as its device
    d = moe.gqa_paged_dims(**GOOD)
    c, s = torch.zeros(100, 2, 64, 128, dtype=torch.uint8), torch.zeros(100, 2, 4)
    assert moe._paged8_caches(c, c.view(torch.float8_e4m3fn), s, s, d, host)[0] == c.data_ptr()
    for bad in (c.to(torch.bfloat16), c[:99], c.transpose(1, 2).contiguous().transpose(1, 2), c[..., :64], c.view(torch.float8_e5m2)):
        with pytest.raises(ValueError):
            moe._paged8_caches(c, bad, s, s, d, host)
    for bad in (s.double(), s[:, :, :2], s.view(100, 8), torch.zeros(100, 4, 2).transpose(1, 2)):
        with pytest.raises(ValueError):
            moe._paged8_caches(c, c, s, bad, d, host)
    with pytest.raises(ValueError):
        moe._paged8_caches(c, c, s, s, d, 0)


def test_kernels_read_tables_coherently():
    """As the 16-bit calls: nothing that a call before may write comes from the read-only data path."""
    for name in ("paged8.cuh", "paged8.cu", "paged8_decode.cu", "paged8_chunk.cu", "paged_chunk.cuh", "rotary.cu"):
        with open(os.path.join(moe.PKG_DIR, "csrc", name)) as f:
            text = f.read()
        for form in ("__ldg(", ".nc.", "__restrict__"):
            assert form not in text, (name, form)


# ---------------------------------------------------------------- rotary positions
ROT = dict(n_heads=16, n_kv_heads=2, head_dim=128, rot_dim=128, n_tokens=37)
FAR = {n: (i + 1) << 24 for i, n in enumerate(("q", "k", "positions", "turns", "n_rows", "q_out", "k_out"))}


def _rotary(lib, d, **kw):
    g = {**FAR, **kw}
    return lib.gqa_rotary(ctypes.byref(d), g["q"], g["k"], g["positions"], g["turns"], g["n_rows"], g["q_out"], g["k_out"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(n_heads=-1), INVALID), (dict(n_heads=0, n_kv_heads=0), INVALID), (dict(rot_dim=0), INVALID), (dict(rot_dim=7), INVALID),
    (dict(rot_dim=130), INVALID), (dict(n_tokens=-1), INVALID), (dict(head_dim=0), INVALID), (dict(amplitude=float("nan")), INVALID),
    (dict(amplitude=float("inf")), INVALID), (dict(head_dim=260, rot_dim=64), UNSUPPORTED), (dict(head_dim=100, rot_dim=64), UNSUPPORTED),
    (dict(n_tokens=1 << 27), UNSUPPORTED), (dict(n_heads=(1 << 19) - 1), UNSUPPORTED), (dict(q_stride=2040), INVALID),
    (dict(q_stride=2052), MISALIGNED),
    (dict(k_out_stride=100), INVALID), (dict(k_stride=1 << 39), UNSUPPORTED)])
def test_rotary_dims_refused(lib, bad, status):
    assert _rotary(lib, moe.gqa_rotary_dims(**{**ROT, **bad})) == status


def test_rotary_fields_and_pointers(lib):
    d = moe.gqa_rotary_dims(**ROT)
    for p in FAR:
        if p != "n_rows":
            assert _rotary(lib, d, **{p: None}) == INVALID, p
        assert _rotary(lib, d, **{p: FAR[p] + (2 if p in ("positions", "n_rows") else 8)}) == MISALIGNED, p
    d.pairs = 2
    assert _rotary(lib, d) == INVALID
    d = moe.gqa_rotary_dims(**ROT)
    d.dtype = 2
    assert _rotary(lib, d) == INVALID
    assert lib.gqa_rotary(None, *[256] * 7, None) == INVALID
    assert _rotary(lib, moe.gqa_rotary_dims(**{**ROT, "n_tokens": 0}), **{p: None for p in FAR}) == 0
    with pytest.raises(KeyError):
        moe.gqa_rotary_dims(**ROT, layout="other")
    with pytest.raises(ValueError):
        moe.gqa_rotary_dims(**{**ROT, "n_tokens": 2**32})


def test_rotary_refuses_outputs_that_overlap(lib):
    """Every output against the inputs and the other output, by one element; rows of one wide buffer beside one another are
    not an overlap, and neither is turning in place (which is not run here: the first row's stride differs)."""
    d = moe.gqa_rotary_dims(**ROT)
    qb, kb = 37 * 16 * 128 * 2, 37 * 2 * 128 * 2
    for out, width in (("q_out", qb), ("k_out", kb)):
        for other, size in (("q", qb), ("k", kb), ("q_out", qb), ("k_out", kb)):
            if other == out:
                continue
            for at in (FAR[other] + size - 16, FAR[other] - width + 16):
                assert _rotary(lib, d, **{out: at}) == INVALID, (out, other)
    # one buffer [T, 18 * 128 + ...]: k's rows behind q's; outputs in the same columns overlap, shifted by a head they do too
    row = (16 + 2 + 16) * 128
    wide = moe.gqa_rotary_dims(**ROT, q_stride=row, k_stride=row, q_out_stride=row)
    q = 1 << 24
    assert _rotary(lib, wide, q=q, k=q + 16 * 128 * 2, q_out=q + 17 * 128 * 2) == INVALID      # k's second head
    assert _rotary(lib, wide, q=q, k=q + 16 * 128 * 2, q_out=q + 128 * 2) == INVALID


@pytest.mark.parametrize("kw", [
    {}, dict(base=1e6), dict(scaling="linear", factor=7.5), dict(scaling="base", factor=4.0), dict(base=1.0),
    dict(scaling="by_parts", factor=16.0, original=8192, base=500000.0), dict(scaling="by_parts", factor=4.0, original=4096, low=0.0, high=2.0)])
@pytest.mark.parametrize("rot", [2, 4, 96, 128, 256])
def test_table_of_frequencies(lib, rot, kw):
    """Each entry within 2^-50 of itself (a handful of double roundings), and half a unit of 2^-64 of a turn."""
    if rot == 2 and kw.get("scaling") == "base":
        with pytest.raises(moe.MoeError):
            moe.gqa_rotary_table(rot, device="cpu", **kw)
        return
    got = moe.gqa_rotary_table(rot, device="cpu", **kw).numpy().view(np.uint64).astype(np.longdouble) / np.longdouble(2) ** 64
    pi = np.longdouble("3.14159265358979323846264338327950288")
    want = Q.frequencies(rot, **kw) / (2 * pi)
    assert got.shape == (rot // 2,) and (np.abs(got - want) <= want * np.longdouble(2) ** -50 + np.longdouble(2) ** -64).all()


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=258), dict(base=0.5), dict(base=float("inf")), dict(base=float("nan")),
    dict(factor=2.0), dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("nan")),
    dict(scaling="by_parts", factor=2.0), dict(scaling="by_parts", factor=2.0, original=4096, low=2.0, high=2.0),
    dict(scaling="by_parts", factor=2.0, original=-1.0), dict(scaling="base", factor=1e300, base=1e300)])
def test_table_refusals(lib, kw):
    with pytest.raises(moe.MoeError):
        moe.gqa_rotary_table(**{**dict(rot_dim=64, device="cpu"), **kw})
    assert lib.gqa_rotary_table(None, 256) == INVALID


def test_table_refusals_of_the_binding(lib):
    for rot in (2**32 + 64, -2):
        with pytest.raises(ValueError):
            moe.gqa_rotary_table(rot, device="cpu")
    with pytest.raises(KeyError):
        moe.gqa_rotary_table(64, scaling="other", device="cpu")


@pytest.mark.parametrize("dtype", [2, -1, 77])
def test_binding_refuses_dims_of_no_type(dtype):
    """As the library itself does, with the same error."""
    import torch
    moe._load_paged_types()
    d, rd = moe.gqa_paged_dims(**GOOD), moe.gqa_rotary_dims(**ROT)
    d.dtype = rd.dtype = dtype
    rows, cache = torch.zeros(37, 16, 128, dtype=torch.bfloat16), torch.zeros(100, 2, 64, 128, dtype=torch.bfloat16)
    for call in (lambda: moe._want8(d), lambda: moe._want_rotary(rd), lambda: moe._paged_caches(cache, cache, d, -1),
                 lambda: moe._paged_rows(rows, 37, 16, 128, 0, dtype, -1, "q")):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert "MOE_ERR_INVALID_ARG" in str(e.value)
