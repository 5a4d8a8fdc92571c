"""Measured cases of the rotary positions and of the paged key/value cache held in 8 bits: queries and keys rotated by
their positions, new keys and values quantised as they are written, a cache read back, and the attention that reads it
(a chunk of new tokens or single tokens per sequence, optionally with a sliding window and leading positions).

An 8-bit cache holds e4m3 codes and one scale for each 16 positions of a page and head, a power of two.

`run` computes each operator from elementary torch operations where `own` is false, and makes the framework's calls
where it is true.  A case's lengths follow from the case alone (`lens` seeds them); values, page order and the like
follow from the seed.
"""
import math
import random

import torch

own = False

GPU = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
BLOCK = 16                    # positions of a scale
LEAST, MOST = -60, 60         # exponents of a scale


def _case(name, op, **kw):
    c = {"name": name, "op": op, "dtype": "bf16", "Hq": 16, "Hkv": 2, "D": 128, "page": 64, "layout": "head",
         "fused": False, "seqs": 1, "chunks": 0, "new": 1, "ctx": 0, "even": False, "pad": 0, "window": 0, "sinks": 0,
         "lens": 1}
    if op == "rotary":
        c.update(rot=128, pairs="half", scaling="none", base=10000.0, factor=1.0, original=0)
    c.update(kw)
    return c


def listed():
    return [
        # Positions of one decode step of a served batch.
        _case("rotary_decode_64", "rotary", seqs=64, ctx=32768, lens=11),
        # Prompt chunks far behind the length that the model was trained at: frequencies scaled part by part, a quarter
        # of each head left as it is, neighbouring dims paired, q and k as views of a fused projection.
        _case("rotary_prompts_far", "rotary", seqs=4, chunks=4, new=2048, ctx=131001, even=True, dtype="fp16", fused=True, rot=96,
              pairs="interleaved", scaling="by_parts", base=500000.0, factor=16.0, original=8192, pad=13),
        # Keys and values of one decode step into their pages.
        _case("append8_decode_64", "append", seqs=64, ctx=4096, lens=13),
        # Keys and values of several prompts, as views of a fused projection, position-major pages.
        _case("append8_prompts_8", "append", seqs=8, chunks=8, new=4096, ctx=2000, dtype="fp16", page=32,
              layout="position", fused=True, lens=36),
        # The prefix of one short conversation, read back for a model whose heads are 64 wide.
        _case("read8_300", "read", seqs=1, chunks=1, new=300, ctx=0, even=True, Hq=8, Hkv=8, D=64, page=16, dtype="fp16"),
        # Whole caches of eight long conversations read back.
        _case("read8_8_long", "read", seqs=8, chunks=8, new=32768, ctx=0, lens=14),
        # One user at a context of 32K.
        _case("decode8_1x32768", "attend", seqs=1, ctx=32767, even=True),
        # A decode step of 64 requests of very different lengths, small pages.
        _case("decode8_64_ragged", "attend", seqs=64, ctx=32768, page=16, dtype="fp16", lens=16),
        # Decoding requests of up to 128K positions that read a window of 4096 and sixteen leading ones.
        _case("window8_decode_32", "attend", seqs=32, ctx=131072, window=4096, sinks=16, lens=21),
        # A later chunk of a long prompt against 32K cached positions.
        _case("chunk8_2048_at_32768", "attend", seqs=1, chunks=1, new=2048, ctx=32768, even=True),
        # Two prompt chunks in one step with 32 decoding requests; odd lengths, q inside a fused projection,
        # position-major pages, rows reserved behind the last sequence.
        _case("mixed8_34_odd", "attend", seqs=34, chunks=2, new=1777, ctx=9001, page=32, dtype="fp16", layout="position",
              fused=True, pad=29, lens=36),
        # Short prompts of a small model: every query head has its own keys, heads of 64.
        _case("prompts8_16_heads_64", "attend", seqs=16, chunks=16, new=300, ctx=1000, Hq=8, Hkv=8, D=64, page=16,
              dtype="fp16", lens=22),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.7e12, w["flops"] / 2.0e15)


def draw(rng):
    top = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("rotary", "append", "read", "attend")}
    while True:
        op = rng.choice(["rotary", "append", "read", "attend", "attend", "attend"])
        hkv, group, d = rng.choice([1, 2, 2, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 8]), rng.choice([64, 128, 128])
        kw = dict(dtype=rng.choice(["bf16", "fp16"]), Hq=hkv * group, Hkv=hkv, D=d, page=rng.choice([16, 32, 64, 128]),
                  layout=rng.choice(["head", "position"]), fused=rng.random() < 0.5, lens=rng.randrange(1 << 30),
                  even=rng.random() < 0.4, pad=rng.choice([0, 0, rng.randrange(1, 64)]))
        if op == "rotary":
            kw.update(seqs=_log(rng, 1, 64), new=_log(rng, 1, 4096), ctx=_log(rng, 1, 131072), pairs=rng.choice(["half", "interleaved"]))
            kw.update(chunks=rng.randrange(0, 9), rot=rng.choice([d, d, d // 2, d // 4, 2 * rng.randrange(1, d // 2 + 1)]))
            kw.update(scaling=rng.choice(["none", "linear", "base", "by_parts"]), base=rng.choice([10000.0, 500000.0, 1e6]))
            if kw["scaling"] != "none":
                kw.update(factor=rng.choice([2.0, 4.0, 7.5, 16.0]), original=rng.choice([2048, 8192]), rot=max(kw["rot"], 4))
        elif op == "append":
            kw.update(seqs=_log(rng, 1, 64), new=_log(rng, 1, 4096), ctx=_log(rng, 1, 4096))
            kw.update(chunks=rng.randrange(0, 9))
        elif op == "read":
            kw.update(seqs=_log(rng, 1, 64), new=_log(rng, 1, 32768), ctx=_log(rng, 1, 4096))
            kw.update(chunks=kw["seqs"])
        else:
            form = rng.choice(["decode", "chunk", "mixed"])
            kw.update(seqs=_log(rng, 1, 64), ctx=_log(rng, 1, 131072), new=1, chunks=0)
            if form != "decode":
                kw.update(new=_log(rng, 2, 4096), seqs=_log(rng, 1, 40))
                kw.update(chunks=kw["seqs"] if form == "chunk" else rng.randrange(1, 4))
            if rng.random() < 0.4:
                kw.update(window=_log(rng, 16, 8192), sinks=rng.choice([0, 1, 4, 16, 100]))
        kw["chunks"] = min(kw["chunks"], kw["seqs"])
        case = _case("drawn", op, **kw)
        del case["name"]
        ctx, new = lengths(case)
        if sum(new) > (1 << 18 if op == "read" else 1 << 16) or (op != "rotary" and (sum(ctx) + sum(new)) * hkv * d > 1 << 29):
            continue
        if _cost(case) <= top[op]:
            return case


def lengths(case):
    """Cached and new positions of each sequence."""
    r = random.Random(case["lens"])
    ctx, new = [], []
    for i in range(case["seqs"]):
        chunk = i < case["chunks"]
        if case["even"]:
            ctx.append(case["ctx"])
            new.append(case["new"] if chunk else 1)
        else:
            ctx.append(_log(r, 1, case["ctx"] + 1) - 1)
            new.append(_log(r, 1, case["new"]) if chunk else 1)
    order = list(range(case["seqs"]))
    r.shuffle(order)                       # chunks stand anywhere among the single tokens
    return [ctx[i] for i in order], [new[i] for i in order]


def _sum_visible(case, c, n):
    """Sum of the visible positions of the tokens at c .. c + n - 1, piece by piece in closed form."""
    w, s = case["window"], case["sinks"]
    tri = lambda a, b: (b * (b - 1) - a * (a - 1)) // 2 + (b - a) if b > a else 0   # sum of p + 1, a <= p < b
    if w == 0:
        return tri(c, c + n)
    full = max(c, min(c + n, w + s))       # positions below w + s see everything
    return tri(c, full) + (c + n - full) * (w + s)


def work(case):
    ctx, new = lengths(case)
    T, B, page, Hq, H, D = sum(new), case["seqs"], case["page"], case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "rotary":
        # Read q and k, write them rotated; six operations a pair.
        return {"bytes": 2 * T * (Hq + H) * D * 2 + 4 * T + 8 * (case["rot"] // 2), "flops": 3 * T * (Hq + H) * case["rot"]}
    if case["op"] == "append":
        # Read the new rows and what the first block of each sequence already holds, write the codes of all these blocks'
        # held positions and their scales.
        held = sum(c % BLOCK for c in ctx)
        blocks = sum(-(-(c + n) // BLOCK) - c // BLOCK for c, n in zip(ctx, new))
        return {"bytes": 2 * H * D * (2 * T + T) + 2 * H * D * held + 2 * H * 4 * blocks + 4 * (blocks + 2 * B), "flops": 0}
    if case["op"] == "read":
        blocks = sum(-(-(c + n) // BLOCK) - c // BLOCK for c, n in zip(ctx, new))
        return {"bytes": 2 * T * H * D * 3 + 2 * H * 4 * blocks + 4 * (blocks * BLOCK // page + 2 * B), "flops": 0}
    pairs, read, pages = 0, 0, 0
    for c, n in zip(ctx, new):
        pairs += _sum_visible(case, c, n)
        lo = max(0, c - case["window"] + 1) if case["window"] else 0
        seen = c + n - lo + min(case["sinks"], lo)
        read += seen
        pages += -(-seen // page)
    return {"bytes": 2 * T * Hq * D * 2 + read * H * D * 2 + -(-read // BLOCK) * H * 2 * 4 + 4 * (pages + 2 * B),
            "flops": 4 * D * Hq * pairs}


def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, within the scales' range."""
    m, x = torch.frexp(amax)               # amax = m 2^x, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax == 0, torch.full_like(e, LEAST), e).clamp(LEAST, MOST)


def _power(e):
    """2^e, by its bits: a power function may be off in the last one."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _frequencies(case):
    """Radians a position of each pair, in 64 bits."""
    i = torch.arange(case["rot"] // 2, dtype=torch.float64)
    base, f = case["base"], case["factor"]
    if case["scaling"] == "base":
        base = base * f ** (case["rot"] / (case["rot"] - 2))
    w = base ** (-2.0 * i / case["rot"])
    if case["scaling"] == "linear":
        w = w / f
    if case["scaling"] == "by_parts":
        keep = ((case["original"] * w / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        w = w * keep + w / f * (1 - keep)
    return w


def _amplitude(case):
    return 1.0 + 0.1 * math.log(case["factor"]) if case["scaling"] == "by_parts" else 1.0


def prepare(case, seed):
    gen = torch.Generator(device=GPU)
    gen.manual_seed(seed)
    ctx, new = lengths(case)
    dt, B, page, Hq, H, D = TYPES[case["dtype"]], case["seqs"], case["page"], case["Hq"], case["Hkv"], case["D"]
    rows, T = sum(new), sum(new) + case["pad"]
    op = case["op"]
    i32 = dict(dtype=torch.int32, device=GPU)
    s = {"case": case, "ctx": ctx, "new": new, "rows": rows, "T": T}
    # Heads differ in how sharply they attend, the dims of keys in size.
    sharp = torch.exp(torch.rand(Hq, generator=gen, device=GPU) * math.log(8.0)) * 0.5
    dims = torch.exp(torch.randn(D, generator=gen, device=GPU) * 0.5)
    if op != "read":
        q = (torch.randn((T, Hq, D), generator=gen, device=GPU) * sharp[None, :, None]).to(dt)
        k = (torch.randn((T, H, D), generator=gen, device=GPU) * dims).to(dt)
        v = torch.randn((T, H, D), generator=gen, device=GPU).to(dt)
        if case["fused"]:                                     # one projection's output holds all three
            qkv = torch.cat([q.reshape(T, -1), k.reshape(T, -1), v.reshape(T, -1)], 1).contiguous()
            q, k, v = (x.view(T, -1, D) for x in qkv.split([Hq * D, H * D, H * D], 1))
        s["q"], s["k"], s["v"] = q, k, v

    if op == "rotary":
        pos = torch.cat([torch.arange(c, c + n, **i32) for c, n in zip(ctx, new)] + [torch.full((case["pad"],), -7, **i32)])
        s["positions"], s["n_rows"] = pos, torch.tensor([rows], **i32)
        s["freq"], s["amplitude"] = _frequencies(case).to(GPU), _amplitude(case)
        s["q_out"], s["k_out"] = torch.zeros((T, Hq, D), dtype=dt, device=GPU), torch.zeros((T, H, D), dtype=dt, device=GPU)
        if own:
            import bit_quantized_expert_gb300 as moe
            s["moe"] = moe
            s["dims"] = moe.gqa_rotary_dims(Hq, H, D, case["rot"], T, layout=case["pairs"], dtype=case["dtype"],
                                            amplitude=s["amplitude"], q_stride=q.stride(0), k_stride=k.stride(0))
            s["table_of_turns"] = moe.gqa_rotary_table(case["rot"], base=case["base"], scaling=case["scaling"],
                                                       factor=case["factor"], original=case["original"])
        return s

    held = [c + n for c, n in zip(ctx, new)]
    max_pages = max(-(-h // page) for h in held) + 1
    counts = [-(-h // page) for h in held]
    num_pages = sum(counts) + 8 + sum(counts) // 16
    # Pages in the order in which a pool hands them out after some time: any order.
    perm = torch.randperm(num_pages, generator=gen, device=GPU).to(torch.int32)
    cnt = torch.tensor(counts, device=GPU)
    col = torch.arange(max_pages, device=GPU)
    base = torch.cumsum(cnt, 0) - cnt
    known = col[None, :] < cnt[:, None]
    s["table"] = torch.where(known, perm[(base[:, None] + col[None, :]).clamp(max=num_pages - 1)],
                             torch.full((), -1, **i32)).contiguous()
    s["new_len"] = torch.tensor(new, **i32)
    s["kv_len"] = torch.tensor(held, **i32)
    s["q_start"] = torch.cat([torch.zeros(1, **i32), torch.cumsum(s["new_len"], 0).to(torch.int32)])
    # A pool that earlier steps have filled: values of its own size in each block, the dims of keys in theirs.
    shape = (num_pages, H, page, D) if case["layout"] == "head" else (num_pages, page, H, D)
    for name, by in (("k", dims), ("v", torch.ones_like(dims))):
        x = torch.randn((num_pages, H, page // BLOCK, BLOCK, D), generator=gen, device=GPU)
        x *= by * torch.exp(torch.randn((num_pages, H, page // BLOCK, 1, 1), generator=gen, device=GPU) * 0.4)
        e = _exponent(x.abs().amax((3, 4)))
        codes = (x * _power(-e)[..., None, None]).to(E4M3).view(torch.uint8).view(num_pages, H, page, D)
        cache = torch.empty(shape, dtype=torch.uint8, device=GPU)
        cache = cache if case["layout"] == "head" else cache.transpose(1, 2)      # always indexed [page, head, offset, D]
        cache.copy_(codes)
        s[name + "_cache"], s[name + "_scale"] = cache, _power(e).contiguous()
        del x, codes
    if op == "read":
        s["k_out"], s["v_out"] = (torch.zeros((T, H, D), dtype=dt, device=GPU) for _ in range(2))
    if op == "attend":
        s["o"] = torch.zeros((T, Hq, D), dtype=dt, device=GPU)
        # What lies behind a sequence's last position was never written: it may hold anything.
        last = s["table"][torch.arange(B, device=GPU), ((s["kv_len"] - 1) // page).long()].long()
        behind = torch.arange(page, device=GPU)[None, :] > ((s["kv_len"] - 1) % page)[:, None]
        which, off = behind.nonzero(as_tuple=True)
        for c in (s["k_cache"], s["v_cache"]):
            c[last[which], :, off] = 0x7F
    if own:
        import bit_quantized_expert_gb300 as moe
        kw = {} if op == "read" else dict(q_stride=q.stride(0), k_stride=k.stride(0), v_stride=v.stride(0))
        s["moe"] = moe
        s["dims"] = moe.gqa_paged_dims(Hq, H, D, page, num_pages, max_pages, B, T, max_new=max(new), window=case["window"],
                                       sinks=case["sinks"], dtype=case["dtype"], cache_strides=s["k_cache"].stride()[:3], **kw)
        s["ws"] = moe.alloc_gqa_paged8_workspace(s["dims"])
    return s


def run(s):
    return {"rotary": _rotary, "append": _append, "read": _read, "attend": _attend}[s["case"]["op"]](s)


def _rotary(s):
    if own:
        s["moe"].gqa_rotary(s["dims"], s["q"], s["k"], s["positions"], s["table_of_turns"], s["q_out"], s["k_out"],
                            n_rows=s["n_rows"])
        return {"q": s["q_out"], "k": s["k_out"]}
    n, rot = s["rows"], s["case"]["rot"]
    angle = s["positions"][:n, None].double() * s["freq"][None, :]
    cos, sin = ((f(angle) * s["amplitude"]).float()[:, None, :] for f in (torch.cos, torch.sin))

    def turn(x, out):
        x = x[:n].float()
        if s["case"]["pairs"] == "half":
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, a * sin + b * cos, x[..., rot:]], -1)
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), x[..., rot:]], -1)
        out[:n] = y.to(out.dtype)
        return out
    return {"q": turn(s["q"], s["q_out"]), "k": turn(s["k"], s["k_out"])}


def _rows(s):
    """Page, offset in the page and position of each row."""
    page, n = s["case"]["page"], s["rows"]
    t = torch.arange(n, device=GPU)
    seq = torch.repeat_interleave(torch.arange(len(s["new"]), device=GPU), s["new_len"].long(), output_size=n)
    pos = (s["kv_len"] - s["q_start"][1:])[seq].long() + t
    return s["table"][seq, pos // page].long(), pos % page, pos


def _append(s):
    page, n = s["case"]["page"], s["rows"]
    if own:
        s["moe"].gqa_paged8_append(s["dims"], s["k"], s["v"], s["table"], s["q_start"], s["kv_len"], s["k_cache"], s["v_cache"],
                                   s["k_scale"], s["v_scale"], s["ws"])
    else:
        pg, off, _ = _rows(s)
        per = page // BLOCK
        block = pg * per + off // BLOCK
        touched, which = torch.unique(block, return_inverse=True)
        first = torch.full_like(touched, BLOCK).scatter_reduce(0, which, off % BLOCK, "amin")     # its first new position
        tp, tb = touched // per, touched % per
        at = torch.arange(BLOCK, device=GPU)
        for name in ("k", "v"):
            cache, scale, x = s[name + "_cache"], s[name + "_scale"], s[name][:n].float()
            H, D = x.shape[1:]
            new_max = torch.zeros((len(touched), H), device=GPU).scatter_reduce(
                0, which[:, None].expand(-1, H), x.abs().amax(2), "amax")
            was = scale[tp, :, tb]
            now = _power(_exponent(new_max))
            now = torch.where((first > 0)[:, None], torch.maximum(now, was), now)
            scale[tp, :, tb] = now
            # What a block holds already, in its new scale (offsets before its first new position), then the new rows.
            offs = (tb * BLOCK)[:, None] + at[None, :]
            old = cache[tp[:, None], :, offs]                                                     # [blocks, 16, H, D]
            moved = (old.view(E4M3).float() * (was / now)[:, None, :, None]).to(E4M3).view(torch.uint8)
            cache[tp[:, None], :, offs] = torch.where((at[None, :] < first[:, None])[..., None, None], moved, old)
            cache[pg, :, off] = (x / now[which][..., None]).to(E4M3).view(torch.uint8)
    return {"k_codes": s["k_cache"].view(E4M3), "v_codes": s["v_cache"].view(E4M3), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _read(s):
    if own:
        s["moe"].gqa_paged8_read(s["dims"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["q_start"],
                                 s["kv_len"], s["k_out"], s["v_out"], s["ws"])
        return {"k": s["k_out"], "v": s["v_out"]}
    n = s["rows"]
    pg, off, _ = _rows(s)
    for name in ("k", "v"):
        x = s[name + "_cache"][pg, :, off].view(E4M3).float() * s[name + "_scale"][pg, :, off // BLOCK][..., None]
        s[name + "_out"][:n] = x.to(s[name + "_out"].dtype)
    return {"k": s["k_out"], "v": s["v_out"]}


def _attend(s):
    if own:
        s["moe"].gqa_paged8_attention(s["dims"], s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                      s["q_start"], s["kv_len"], s["o"], s["ws"])
        return s["o"]
    case = s["case"]
    page, H, D, W, S = case["page"], case["Hkv"], case["D"], case["window"], case["sinks"]
    G, o, row = case["Hq"] // H, torch.zeros_like(s["o"]), 0
    for b, (c, n) in enumerate(zip(s["ctx"], s["new"])):
        L = c + n
        lo = max(0, c - W + 1) if W else 0                # first position that a window reaches
        first = min(S, lo) if W else 0

        # Keys and values of the pages that hold visible positions, in their order, in 32 bits.
        def gather(name):
            def part(a, e):
                pages = s["table"][b, a // page:-(-e // page)].long()
                x = s[name + "_cache"][pages].view(E4M3).float().unflatten(2, (-1, BLOCK)) * s[name + "_scale"][pages][..., None, None]
                x = x.flatten(2, 3).transpose(0, 1).reshape(H, -1, D)
                return x[:, a - a // page * page:][:, :e - a]
            return part(lo, L) if first == 0 else torch.cat([part(0, first), part(lo, L)], 1)
        K, V = gather("k"), gather("v")
        j = torch.arange(lo, L, device=GPU)
        if first:
            j = torch.cat([torch.arange(first, device=GPU), j])
        q = s["q"][row:row + n].float().view(n, H, G, D).transpose(0, 1)          # [H, n, G, D]
        step = max(1, (1 << 28) // (H * G * K.shape[1]))
        for t in range(0, n, step):
            m = min(step, n - t)
            x = q[:, t:t + m].reshape(H, m * G, D) @ K.transpose(1, 2) / math.sqrt(D)
            if n > 1 or W:
                p = torch.arange(c + t, c + t + m, device=GPU)[:, None]
                see = j[None, :] <= p
                if W:
                    see &= (j[None, :] > p - W) | (j[None, :] < S)
                x = x.view(H, m, G, -1).masked_fill(~see[None, :, None, :], float("-inf")).view(H, m * G, -1)
            e = torch.exp(x - x.amax(-1, keepdim=True))
            y = (e @ V) / e.sum(-1, keepdim=True)
            o[row + t:row + t + m] = y.view(H, m, G, D).transpose(0, 1).reshape(m, H * G, D).to(o.dtype)
        row += n
    return o


def exact(case, seed):
    """The definitions in 64 bits: one sequence at a time, and in the attention one query head."""
    global own
    before, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = before
    return {"rotary": _exact_rotary, "append": _exact_append, "read": _exact_read, "attend": _exact_attend}[case["op"]](s)


def _exact_rotary(s):
    """Each pair as a complex number, turned."""
    case, n = s["case"], s["rows"]
    rot = case["rot"]
    at = torch.tensor([p for c, m in zip(s["ctx"], s["new"]) for p in range(c, c + m)], dtype=torch.float64, device=GPU)
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=GPU)
    f = case["factor"]
    base = case["base"] * (f ** (rot / (rot - 2)) if case["scaling"] == "base" else 1)
    w = torch.exp(-i / rot * math.log(base))
    if case["scaling"] == "linear":
        w = w / f
    elif case["scaling"] == "by_parts":            # kept above 32 turns of the original length, stretched below one
        turns = case["original"] * w / (2 * math.pi)
        part = torch.clamp((turns - 1) / 31, 0, 1)
        w = (1 - part) * w / f + part * w
    spin = torch.polar(torch.full((n, rot // 2), _amplitude(case), dtype=torch.float64, device=GPU), at[:, None] * w)
    out = {}
    for name in ("q", "k"):
        x, y = s[name].double(), torch.zeros(s[name].shape, dtype=torch.float64, device=GPU)
        lo, hi = (slice(0, rot // 2), slice(rot // 2, rot)) if case["pairs"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
        z = torch.complex(x[:n, :, lo].contiguous(), x[:n, :, hi].contiguous()) * spin[:, None, :]
        y[:n, :, lo], y[:n, :, hi], y[:n, :, rot:] = z.real, z.imag, x[:n, :, rot:]
        out[name] = y
    return out


def _nearest_e4m3(y):
    """y rounded to 1 + 3 bits, half to even, steps of 2^-9 below 2^-6."""
    _, x = torch.frexp(y)
    step = _double_power(torch.clamp(x, min=-5) - 4)
    return torch.round(y / step) * step


def _double_power(e):
    return (e.long() + 1023).bitwise_left_shift(52).view(torch.float64)


def _exact_append(s):
    """Sequence by sequence, the blocks of 16 that get new positions side by side."""
    case = s["case"]
    page, out, row = case["page"], {}, 0
    values = {n: s[n + "_cache"].contiguous().view(E4M3).double() for n in ("k", "v")}
    scales = {n: s[n + "_scale"].double() for n in ("k", "v")}
    for b, (c, m) in enumerate(zip(s["ctx"], s["new"])):
        lo, hi = c // BLOCK * BLOCK, -(-(c + m) // BLOCK) * BLOCK
        pos = torch.arange(lo, hi, device=GPU)
        pg, off = s["table"][b].long()[pos.div(page, rounding_mode="floor")], pos.remainder(page)
        fresh = (pos >= c) & (pos < c + m)
        kept = pos < c
        for n in ("k", "v"):
            have = values[n][pg, :, off]                                                      # [positions, H, D]
            was = scales[n][pg[::BLOCK], :, off[::BLOCK] // BLOCK]                            # [blocks, H]
            x = torch.zeros_like(have)
            x[fresh] = s[n][row:row + m].double()
            top = x.abs().unflatten(0, (-1, BLOCK)).amax((1, 3))
            power = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 448)).clamp(LEAST, MOST)
            power = torch.where(_double_power(power - 1) * 448 >= top, power - 1, power).clamp(LEAST, MOST)
            power = torch.where(_double_power(power) * 448 < top, power + 1, power).clamp(LEAST, MOST)
            now = _double_power(power)
            now[0] = torch.maximum(now[0], was[0]) if c > lo else now[0]
            each, before = now.repeat_interleave(BLOCK, 0)[..., None], was.repeat_interleave(BLOCK, 0)[..., None]
            y = torch.where(kept[:, None, None], _nearest_e4m3(have * before / each), have)
            values[n][pg, :, off] = torch.where(fresh[:, None, None], _nearest_e4m3(x / each), y)
            scales[n][pg[::BLOCK], :, off[::BLOCK] // BLOCK] = now
        row += m
    for n in ("k", "v"):
        out[n + "_codes"], out[n + "_scale"] = values[n], scales[n]
    return out


def _exact_read(s):
    page, row = s["case"]["page"], 0
    out = {n: torch.zeros(s[n + "_out"].shape, dtype=torch.float64, device=GPU) for n in ("k", "v")}
    for b, (c, m) in enumerate(zip(s["ctx"], s["new"])):
        pos = torch.arange(c, c + m, device=GPU)
        pg, off = s["table"][b].long()[pos.div(page, rounding_mode="floor")], pos.remainder(page)
        for n in ("k", "v"):
            for h in range(s["case"]["Hkv"]):
                codes = s[n + "_cache"][:, h][pg, off].view(E4M3).double()
                out[n][row:row + m, h] = codes * s[n + "_scale"][:, h][pg, off // BLOCK].double()[:, None]
        row += m
    return out


def _exact_attend(s):
    case = s["case"]
    page, D, G = case["page"], case["D"], case["Hq"] // case["Hkv"]
    if work(case)["flops"] > 4e12:
        return None
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=GPU)
    begin = 0
    for b in range(case["seqs"]):
        n, L = s["new"][b], s["ctx"][b] + s["new"][b]
        pos = torch.arange(L, device=GPU)
        if case["window"]:
            pos = pos[(pos > s["ctx"][b] - case["window"]) | (pos < case["sinks"])]
        pg, off = s["table"][b].long()[pos.div(page, rounding_mode="floor")], pos.remainder(page)
        for g in range(case["Hkv"]):
            keys, vals = (s[m + "_cache"][pg, g, off].view(E4M3).double() * s[m + "_scale"][pg, g, off // BLOCK].double()[:, None]
                          for m in ("k", "v"))
            for h in range(g * G, (g + 1) * G):
                for t0 in range(0, n, 1024):
                    t1 = min(n, t0 + 1024)
                    mine = torch.arange(L - n + t0, L - n + t1, device=GPU)
                    logit = torch.einsum("td,jd->tj", s["q"][begin + t0:begin + t1, h].double(), keys) * D ** -0.5
                    hidden = pos.unsqueeze(0) > mine.unsqueeze(1)
                    if case["window"]:
                        near = mine.unsqueeze(1) - pos.unsqueeze(0) < case["window"]
                        hidden |= ~(near | (pos.unsqueeze(0) < case["sinks"]))
                    logit[hidden] = -math.inf
                    o[begin + t0:begin + t1, h] = torch.softmax(logit, 1) @ vals
        begin += n
    return o
