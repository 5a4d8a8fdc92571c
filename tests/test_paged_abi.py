"""Host-side refusals of the paged calls (include/gqa_paged.h): every call below returns from the argument
checks before any CUDA work is enqueued, so no GPU is needed."""
import ctypes
import os

import pytest

import bit_quantized_expert_gb300 as moe


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from bit_quantized_expert_gb300 import build
        build.build()
    return moe.load_library()


GOOD = dict(n_heads=16, n_kv_heads=2, head_dim=128, page_size=64, num_pages=100, max_pages=20, n_seqs=4, n_tokens=37)


def _calls(lib):
    """The three calls with every pointer given by name (all good by default)."""
    def nb(d):
        return lib.gqa_paged_workspace_bytes(ctypes.byref(moe.gqa_paged_dims(**GOOD)))

    def plan(d, **kw):
        g = lambda n: kw.get(n, 256)
        return lib.gqa_paged_plan(ctypes.byref(d), g("ctx"), g("new"), g("free"), kw.get("cap", 100), g("n_free"),
                                  g("table"), g("q_start"), g("kv_len"), g("positions"), g("slots"), g("n_out"), g("ws"),
                                  kw.get("nb", nb(d)), None)

    def append(d, **kw):
        g = lambda n: kw.get(n, 256)
        return lib.gqa_paged_append(ctypes.byref(d), g("k"), g("v"), g("slots"), g("q_start"), g("kc"), g("vc"), g("ws"),
                                    kw.get("nb", nb(d)), None)

    def attention(d, **kw):
        g = lambda n: kw.get(n, 256)
        return lib.gqa_paged_attention(ctypes.byref(d), g("q"), g("kc"), g("vc"), g("table"), g("q_start"), g("kv_len"),
                                       g("o"), g("ws"), kw.get("nb", nb(d)), None)

    return {"plan": (plan, ("ctx", "new", "free", "n_free", "table", "q_start", "kv_len", "slots", "n_out", "ws")),
            "append": (append, ("k", "v", "slots", "q_start", "kc", "vc", "ws")),
            "attention": (attention, ("q", "kc", "vc", "table", "q_start", "kv_len", "o", "ws"))}


@pytest.mark.parametrize("name", ["plan", "append", "attention"])
def test_pointers_and_workspace(lib, name):
    """1 for a null pointer, 3 for one off its alignment (4 bytes for the int32 tables, 16 for all else),
    4 for a short workspace."""
    call, pointers = _calls(lib)[name]
    d = moe.gqa_paged_dims(**GOOD)
    for p in pointers:
        assert call(d, **{p: None}) == 1, p
        assert call(d, **{p: 264 if p in ("q", "k", "v", "kc", "vc", "o", "ws") else 258}) == 3, p
    assert call(d, nb=lib.gqa_paged_workspace_bytes(ctypes.byref(d)) - 1) == 4
    if name == "plan":
        assert call(d, positions=258) == 3 and call(d, cap=-1) == 1
        assert call(d, free=None, cap=0, ws=None) == 1 and call(d, free=None, cap=0, nb=0) == 4


def test_plan_refuses_outputs_that_overlap(lib):
    """Every output against every input and every other output, by its last or first 4 bytes."""
    d = moe.gqa_paged_dims(**GOOD)
    B, T, M, cap = d.n_seqs, d.n_tokens, d.max_pages, 100
    size = dict(ctx=B, new=B, free=cap, n_free=1, table=B * M, q_start=B + 1, kv_len=B, positions=T, slots=T, n_out=1)
    apart = {n: 4096 * (i + 1) for i, n in enumerate(size)}
    plan = _calls(lib)["plan"][0]
    for out in ("table", "q_start", "kv_len", "positions", "slots", "n_out"):
        for other in size:
            if other == out:
                continue
            ends = [apart[other] + 4 * (size[other] - 1), apart[other] - 4 * (size[out] - 1)]
            for at in ends:
                if (out, other) == ("n_out", "n_free"):
                    continue   # the same counter is allowed
                assert plan(d, **{**apart, out: at, "ws": 1 << 20}) == 1, (out, other)


INVALID, UNSUPPORTED, MISALIGNED = 1, 2, 3


@pytest.mark.parametrize("bad,status", [
    (dict(n_heads=0), INVALID), (dict(n_kv_heads=0), INVALID), (dict(n_heads=15), INVALID), (dict(page_size=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(n_seqs=-1), INVALID), (dict(n_tokens=-1), INVALID),
    (dict(max_new=-1), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED), (dict(n_heads=18), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED), (dict(n_seqs=4097), UNSUPPORTED),
    (dict(num_pages=1 << 24, page_size=128), UNSUPPORTED), (dict(num_pages=1 << 24), UNSUPPORTED),
    (dict(max_pages=1 << 25), UNSUPPORTED), (dict(max_pages=(1 << 24) + 1), UNSUPPORTED), (dict(n_tokens=1 << 27), UNSUPPORTED),
    (dict(q_stride=2047), INVALID), (dict(q_stride=2052), MISALIGNED), (dict(k_stride=248), INVALID),
    (dict(v_stride=260), MISALIGNED), (dict(o_stride=1 << 39), UNSUPPORTED), (dict(q_stride=-2048), INVALID),
    (dict(cache_strides=(16384, 8192, 132)), MISALIGNED), (dict(cache_strides=(16384, 8192, 64)), INVALID),
    (dict(cache_strides=(16384, 8064, 128)), INVALID),      # heads overlap
    (dict(cache_strides=(16256, 8192, 128)), INVALID),      # pages overlap
    (dict(cache_strides=(16384, 128, 128)), INVALID)])      # heads and positions at one address
def test_dims_refused(lib, bad, status):
    if "n_heads" in bad and bad["n_heads"] == 18:
        bad = dict(n_heads=18, n_kv_heads=2)
    d = moe.gqa_paged_dims(**{**GOOD, **bad})
    assert lib.gqa_paged_workspace_bytes(ctypes.byref(d)) == 0
    for call, _ in _calls(lib).values():
        assert call(d) == status
        # the dims are looked at first
        assert call(d, ws=None) == status
    with pytest.raises(moe.MoeError):
        moe.alloc_gqa_paged_workspace(d)


def test_unknown_type_refused(lib):
    d = moe.gqa_paged_dims(**GOOD)
    d.dtype = 2
    assert lib.gqa_paged_workspace_bytes(ctypes.byref(d)) == 0
    with pytest.raises(KeyError):
        moe.gqa_paged_dims(**GOOD, dtype="fp8")


def test_null_dims(lib):
    assert lib.gqa_paged_workspace_bytes(None) == 0
    assert lib.gqa_paged_attention(None, *[256] * 8, 1 << 30, None) == 1


@pytest.mark.parametrize("extra", [
    {}, dict(max_pages=1 << 24), dict(page_size=16), dict(page_size=128), dict(head_dim=64), dict(n_heads=2), dict(dtype="fp16"), dict(max_new=1),
    dict(window=100, sinks=4), dict(window=2**31 - 1, sinks=2**31 - 1), dict(q_stride=2560, k_stride=2560, v_stride=2560),
    dict(cache_strides=(16384, 128, 256)),              # position-major pages
    dict(cache_strides=(32768, 8192, 128)),             # keys and values interleaved page by page
    dict(cache_strides=(128, 12800, 25600))])           # pages innermost
def test_dims_accepted(lib, extra):
    d = moe.gqa_paged_dims(**{**GOOD, **extra})
    assert lib.gqa_paged_workspace_bytes(ctypes.byref(d)) >= 256


@pytest.mark.parametrize("name", ["plan", "append", "attention"])
def test_nothing_to_do(lib, name):
    """No sequences, and (but for the plan, which still writes the starts and lengths) no tokens."""
    call, pointers = _calls(lib)[name]
    none = {p: None for p in pointers}
    assert call(moe.gqa_paged_dims(**{**GOOD, "n_seqs": 0}), **none) == 0
    assert call(moe.gqa_paged_dims(**{**GOOD, "n_tokens": 0}), **none) == (1 if name == "plan" else 0)


def test_binding_refuses_host_tensors():
    """The binding raises before it calls the library (tensors that are not on the device of the call)."""
    import torch
    moe._load_paged_types()
    d, x = moe.gqa_paged_dims(**GOOD), torch.zeros(37, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe._paged_ints(torch.zeros(8, dtype=torch.int32), 4, 0, "x")
    with pytest.raises(ValueError):
        moe._paged_rows(x, 37, 16, 128, 0, 0, 0, "q")
    with pytest.raises(ValueError):
        moe._paged_caches(*[torch.zeros(100, 2, 64, 128, dtype=torch.bfloat16)] * 2, d, 0)
    with pytest.raises(ValueError):
        moe._paged_workspace(torch.zeros(1024, dtype=torch.uint8), 0)


def test_kernels_read_tables_coherently():
    """The paged kernels start while the call before them still runs, and the tables and rows that it writes must not come
    from the read-only data path, which promises nothing about data that changes while the kernel runs."""
    for name in ("paged.cuh", "paged.cu", "paged_decode.cu", "paged_chunk.cu"):
        with open(os.path.join(moe.PKG_DIR, "csrc", name)) as f:
            text = f.read()
        for form in ("__ldg(", ".nc.", "__restrict__"):
            assert form not in text, (name, form)


@pytest.mark.parametrize("bad", [dict(window=2**32 + 64), dict(window=2**31), dict(sinks=2**32), dict(n_tokens=2**32 + 37),
                                 dict(max_new=2**32 + 1), dict(page_size=-2**31 - 1), dict(q_stride=2**64 + 2048),
                                 dict(cache_strides=(2**64 + 16384, 8192, 128))])
def test_dims_that_do_not_fit_their_fields(bad):
    """A number past its field's range is refused, not taken modulo 2^32 or 2^64."""
    with pytest.raises(ValueError):
        moe.gqa_paged_dims(**{**GOOD, **bad})


def test_binding_refuses_tables_of_other_widths():
    """A block table whose rows are not max_pages wide would be read across its rows."""
    import torch
    moe._load_paged_types()
    host = -1   # what a host tensor gives as its device
    table = torch.zeros(4, 20, dtype=torch.int32)
    assert moe._paged_table(table, 4, 20, host) == table.data_ptr()
    assert moe._paged_table(table, 3, 20, host) == table.data_ptr()
    assert moe._paged_table(table.view(-1), 4, 20, host) == table.data_ptr()
    for bad in (torch.zeros(4, 32, dtype=torch.int32), torch.zeros(8, 10, dtype=torch.int32), table[:3], table.t(),
                torch.zeros(2, 2, 20, dtype=torch.int32), table.long(), torch.zeros(79, dtype=torch.int32)):
        with pytest.raises(ValueError):
            moe._paged_table(bad, 4, 20, host)
