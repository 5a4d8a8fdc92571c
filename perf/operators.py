"""Measured cases of the paged key/value cache: its plan (block tables and slot maps from request
lengths), the append of new keys and values, and the attention that reads it (a chunk of new tokens
or single tokens per sequence, optionally with a sliding window and leading positions that stay
visible).

`run` computes each operator from elementary torch operations where `own` is false, and makes the
framework's calls where it is true.  A case's lengths follow from the case alone (`lens` seeds
them); values, page order and the free list follow from the seed.
"""
import math
import random

import torch

own = False

GPU = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(name, op, **kw):
    c = {"name": name, "op": op, "dtype": "bf16", "Hq": 16, "Hkv": 2, "D": 128, "page": 64, "layout": "head",
         "fused": False, "seqs": 1, "chunks": 0, "new": 1, "ctx": 0, "even": False, "pad": 0, "window": 0, "sinks": 0,
         "lens": 1}
    c.update(kw)
    return c


def listed():
    return [
        # Tables of one decode step of a served batch: one new token a sequence, most need no page.
        _case("plan_decode_64", "plan", seqs=64, ctx=32768, lens=11),
        # Tables of a large continuous batch with prompt chunks beside single tokens, small pages,
        # rows reserved behind the last sequence.
        _case("plan_mixed_1024", "plan", seqs=1024, chunks=96, new=1000, ctx=16384, page=16, pad=37, lens=12),
        # Keys and values of one decode step into their pages.
        _case("append_decode_64", "append", seqs=64, ctx=4096, lens=13),
        # Keys and values of several prompts, as views of a fused projection, position-major pages.
        _case("append_prompts_8", "append", seqs=8, chunks=8, new=4096, ctx=2000, dtype="fp16", page=32,
              layout="position", fused=True, lens=36),
        # One user at a context of 32K: the decode step of the engine this framework serves.
        _case("decode_1x32768", "attend", seqs=1, ctx=32767, even=True),
        # A decode step of 64 requests of very different lengths, small pages.
        _case("decode_64_ragged", "attend", seqs=64, ctx=32768, page=16, dtype="fp16", lens=16),
        # The first chunk of a prompt (the framework's prefill length), nothing cached.
        _case("prompt_512", "attend", seqs=1, chunks=1, new=512, ctx=0, even=True),
        # A later chunk of a long prompt against 32K cached positions.
        _case("chunk_2048_at_32768", "attend", seqs=1, chunks=1, new=2048, ctx=32768, even=True),
        # Two prompt chunks in one step with 32 decoding requests; odd lengths, q inside a fused
        # projection, position-major pages, rows reserved behind the last sequence.
        _case("mixed_34_odd", "attend", seqs=34, chunks=2, new=1777, ctx=9001, page=32, dtype="fp16", layout="position",
              fused=True, pad=29, lens=36),
        # A long chunk with a window of 1024 positions and four leading positions kept visible.
        _case("window_chunk_4096", "attend", seqs=1, chunks=1, new=4096, ctx=28001, even=True, window=1024, sinks=4),
        # Decoding requests of up to 128K positions that read a window of 4096 and sixteen leading ones.
        _case("window_decode_32", "attend", seqs=32, ctx=131072, window=4096, sinks=16, lens=21),
        # Short prompts of a small model: every query head has its own keys, heads of 64.
        _case("prompts_16_heads_64", "attend", seqs=16, chunks=16, new=300, ctx=1000, Hq=8, Hkv=8, D=64, page=16,
              dtype="fp16", lens=22),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.7e12, w["flops"] / 2.0e15)


def draw(rng):
    top = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("plan", "append", "attend")}
    while True:
        op = rng.choice(["plan", "append", "attend", "attend", "attend", "attend"])
        hkv, group, d = rng.choice([1, 2, 2, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 8]), rng.choice([64, 128, 128])
        kw = dict(dtype=rng.choice(["bf16", "fp16"]), Hq=hkv * group, Hkv=hkv, D=d, page=rng.choice([16, 32, 64, 128]),
                  layout=rng.choice(["head", "position"]), fused=rng.random() < 0.5, lens=rng.randrange(1 << 30),
                  even=rng.random() < 0.4, pad=rng.choice([0, 0, rng.randrange(1, 64)]))
        if op == "plan":
            kw.update(seqs=_log(rng, 1, 1024), new=_log(rng, 1, 1000), ctx=_log(rng, 1, 32768))
            kw.update(chunks=_log(rng, 1, 96))
        elif op == "append":
            kw.update(seqs=_log(rng, 1, 64), new=_log(rng, 1, 4096), ctx=_log(rng, 1, 4096))
            kw.update(chunks=rng.randrange(0, 9))
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
        if sum(new) > 1 << 16 or (op != "plan" and (sum(ctx) + sum(new)) * hkv * d > 1 << 29):
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


def _visible(case, p):
    """Positions that the token at position p sees."""
    if case["window"] == 0 or case["window"] >= p + 1:
        return p + 1
    return case["window"] + min(case["sinks"], p + 1 - case["window"])


def _sum_visible(case, c, n):
    """Sum of _visible over the positions c .. c + n - 1, piece by piece in closed form."""
    w, s = case["window"], case["sinks"]
    tri = lambda a, b: (b * (b - 1) - a * (a - 1)) // 2 + (b - a) if b > a else 0   # sum of p + 1, a <= p < b
    if w == 0:
        return tri(c, c + n)
    full = max(c, min(c + n, w + s))       # positions below w + s see everything
    return tri(c, full) + (c + n - full) * (w + s)


def work(case):
    ctx, new = lengths(case)
    T, B, page, H, D = sum(new), case["seqs"], case["page"], case["Hkv"], case["D"]
    if case["op"] == "plan":
        fresh = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(ctx, new))
        # Read the lengths, the taken pages and one known page a sequence; write the starts, the
        # lengths, the new table entries, the positions and the slots.
        return {"bytes": 4 * (2 * B + fresh + B + (B + 1) + B + fresh + 2 * T + 2), "flops": 0}
    if case["op"] == "append":
        return {"bytes": 4 * T * H * D * 2 + 4 * T, "flops": 0}
    pairs, read, pages = 0, 0, 0
    for c, n in zip(ctx, new):
        pairs += _sum_visible(case, c, n)
        lo = max(0, c - case["window"] + 1) if case["window"] else 0
        seen = c + n - lo + min(case["sinks"], lo)
        read += seen
        pages += -(-seen // page)
    return {"bytes": 2 * T * case["Hq"] * D * 2 + read * H * D * 2 * 2 + 4 * (pages + 2 * B),
            "flops": 4 * D * case["Hq"] * pairs}


def prepare(case, seed):
    gen = torch.Generator(device=GPU)
    gen.manual_seed(seed)
    ctx, new = lengths(case)
    dt, B, page, Hq, H, D = TYPES[case["dtype"]], case["seqs"], case["page"], case["Hq"], case["Hkv"], case["D"]
    rows, T = sum(new), sum(new) + case["pad"]
    op = case["op"]
    held = ctx if op == "plan" else [c + n for c, n in zip(ctx, new)]
    max_pages = max(-(-(c + n) // page) for c, n in zip(ctx, new)) + 1
    counts = [-(-h // page) for h in held]
    fresh = sum(-(-(c + n) // page) for c, n in zip(ctx, new)) - sum(counts)
    num_pages = sum(counts) + fresh + 8 + sum(counts) // 16
    i32 = dict(dtype=torch.int32, device=GPU)

    # Pages in the order in which a pool hands them out after some time: any order.
    perm = torch.randperm(num_pages, generator=gen, device=GPU).to(torch.int32)
    cnt = torch.tensor(counts, device=GPU)
    col = torch.arange(max_pages, device=GPU)
    base = torch.cumsum(cnt, 0) - cnt
    known = col[None, :] < cnt[:, None]
    table = torch.where(known, perm[(base[:, None] + col[None, :]).clamp(max=num_pages - 1)], torch.full((), -1, **i32))
    s = {"case": case, "ctx": ctx, "new": new, "rows": rows, "T": T, "table": table.contiguous(),
         "ctx_len": torch.tensor(ctx, **i32), "new_len": torch.tensor(new, **i32)}

    if op == "plan":
        s["free"] = perm[sum(counts):].contiguous()
        s["n_free"] = torch.tensor([num_pages - sum(counts)], **i32)
        s["table_before"] = s["table"].clone()
        s["out"] = {"q_start": torch.zeros(B + 1, **i32), "kv_len": torch.zeros(B, **i32),
                    "positions": torch.full((T,), -7, **i32), "slots": torch.full((T,), -7, **i32),
                    "n_free": torch.zeros(1, **i32)}
    else:
        s["kv_len"] = s["ctx_len"] + s["new_len"]
        s["q_start"] = torch.cat([torch.zeros(1, **i32), torch.cumsum(s["new_len"], 0).to(torch.int32)])
        shape = (num_pages, H, page, D) if case["layout"] == "head" else (num_pages, page, H, D)
        caches = [torch.randn(shape, generator=gen, device=GPU, dtype=dt) for _ in range(2)]
        if case["layout"] != "head":
            caches = [c.transpose(1, 2) for c in caches]      # always indexed [page, head, offset, D]
        s["k_cache"], s["v_cache"] = caches
        # Heads differ in how sharply they attend.
        scale = torch.exp(torch.rand(Hq, generator=gen, device=GPU) * math.log(8.0)) * 0.5
        q = (torch.randn((T, Hq, D), generator=gen, device=GPU) * scale[None, :, None]).to(dt)
        k = torch.randn((T, H, D), generator=gen, device=GPU).to(dt)
        v = torch.randn((T, H, D), generator=gen, device=GPU).to(dt)
        if case["fused"]:                                     # one projection's output holds all three
            qkv = torch.cat([q.reshape(T, -1), k.reshape(T, -1), v.reshape(T, -1)], 1).contiguous()
            q, k, v = (x.view(T, -1, D) for x in qkv.split([Hq * D, H * D, H * D], 1))
        s["q"], s["k"], s["v"] = q, k, v
        if op == "append":
            pos = torch.cat([torch.arange(c, c + n, device=GPU) for c, n in zip(ctx, new)])
            seq = torch.repeat_interleave(torch.arange(B, device=GPU), s["new_len"].long())
            slots = table[seq, pos // page] * page + pos % page
            s["slots"] = torch.cat([slots.to(torch.int32), torch.full((case["pad"],), -7, **i32)])
        else:
            s["o"] = torch.zeros((T, Hq, D), dtype=dt, device=GPU)
            # What lies behind a sequence's last position was never written: it may hold anything.
            last = table[torch.arange(B, device=GPU), ((s["kv_len"] - 1) // page).long()].long()
            behind = torch.arange(page, device=GPU)[None, :] > ((s["kv_len"] - 1) % page)[:, None]
            which, off = behind.nonzero(as_tuple=True)
            for c in caches:
                c[last[which], :, off] = float("nan")
    if own:
        import bit_quantized_expert_gb300 as moe
        kw = {}
        if op != "plan":
            kw = dict(cache_strides=s["k_cache"].stride()[:3], q_stride=s["q"].stride(0), k_stride=s["k"].stride(0),
                      v_stride=s["v"].stride(0))
        s["moe"] = moe
        s["dims"] = moe.gqa_paged_dims(Hq, H, D, page, num_pages, max_pages, B, T, max_new=max(new),
                                       window=case["window"], sinks=case["sinks"], dtype=case["dtype"], **kw)
        s["ws"] = moe.alloc_gqa_paged_workspace(s["dims"])
    return s


def run(s):
    return {"plan": _plan, "append": _append, "attend": _attend}[s["case"]["op"]](s)


def _plan(s):
    page, out = s["case"]["page"], s["out"]
    if own:
        s["moe"].gqa_paged_plan(s["dims"], s["ctx_len"], s["new_len"], s["free"], s["n_free"], s["table"],
                                out["q_start"], out["kv_len"], out["positions"], out["slots"], out["n_free"], s["ws"])
        return {"table": s["table"], **out}
    ctx, new, table, T, B = s["ctx_len"].long(), s["new_len"].long(), s["table_before"], s["T"], s["case"]["seqs"]
    start = torch.cumsum(new, 0) - new
    total = start[-1] + new[-1]
    old, held = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    need = held - old
    base = torch.cumsum(need, 0) - need
    col = torch.arange(table.shape[1], device=GPU)[None, :]
    take = s["n_free"].long() - 1 - (base[:, None] + col - old[:, None])
    taken = s["free"][take.clamp(0, s["free"].numel() - 1)]
    table = torch.where((col >= old[:, None]) & (col < held[:, None]), taken, table)
    t = torch.arange(T, device=GPU)
    seq = torch.searchsorted(start + new, t, right=True).clamp(max=B - 1)
    pos = ctx[seq] + t - start[seq]
    slot = table[seq, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    live = t < total
    return {"table": table, "q_start": torch.cat([start, total[None]]).int(), "kv_len": (ctx + new).int(),
            "positions": torch.where(live, pos.int(), out["positions"]),
            "slots": torch.where(live, slot.int(), out["slots"]),
            "n_free": (s["n_free"].long() - need.sum()).int()}


def _append(s):
    if own:
        s["moe"].gqa_paged_append(s["dims"], s["k"], s["v"], s["slots"], s["q_start"], s["k_cache"], s["v_cache"], s["ws"])
    else:
        n, page = s["rows"], s["case"]["page"]
        slot = s["slots"][:n].long()
        s["k_cache"][slot // page, :, slot % page] = s["k"][:n]
        s["v_cache"][slot // page, :, slot % page] = s["v"][:n]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attend(s):
    if own:
        s["moe"].gqa_paged_attention(s["dims"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["kv_len"],
                                     s["o"], s["ws"])
        return s["o"]
    case = s["case"]
    page, H, D, W, S = case["page"], case["Hkv"], case["D"], case["window"], case["sinks"]
    G, o, row = case["Hq"] // H, torch.zeros_like(s["o"]), 0
    for b, (c, n) in enumerate(zip(s["ctx"], s["new"])):
        L = c + n
        lo = max(0, c - W + 1) if W else 0                # first position that a window reaches
        first = min(S, lo) if W else 0
        # Keys and values of the pages that hold visible positions, in their order, in 32 bits.
        def gather(cache):
            def part(a, e):
                pages = s["table"][b, a // page:-(-e // page)].long()
                x = cache[pages].transpose(0, 1).reshape(H, -1, D)
                return x[:, a - a // page * page:][:, :e - a].float()
            return part(lo, L) if first == 0 else torch.cat([part(0, first), part(lo, L)], 1)
        K, V = gather(s["k_cache"]), gather(s["v_cache"])
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
    """The definition in 64 bits: one query head and one sequence at a time, positions fetched
    through their slots."""
    global own
    before, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = before
    if case["op"] == "plan":
        return _exact_plan(s)
    page, D, G = case["page"], case["D"], case["Hq"] // case["Hkv"]
    if case["op"] == "append":
        out = {}
        for name, x in (("k_cache", s["k"]), ("v_cache", s["v"])):
            y = s[name].double()
            flat = s["slots"][:s["rows"]].long()
            for h in range(case["Hkv"]):
                y[flat.div(page, rounding_mode="floor"), h, flat.remainder(page)] = x[:s["rows"], h].double()
            out[name] = y
        return out
    if work(case)["flops"] > 4e12:
        return None
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=GPU)
    begin = 0
    for b in range(case["seqs"]):
        n, L = s["new"][b], s["ctx"][b] + s["new"][b]
        pos = torch.arange(L, device=GPU)
        if case["window"]:
            pos = pos[(pos > s["ctx"][b] - case["window"]) | (pos < case["sinks"])]
        at = s["table"][b].long()[pos.div(page, rounding_mode="floor")], pos.remainder(page)
        for g in range(case["Hkv"]):
            keys = s["k_cache"][at[0], g, at[1]].double()
            vals = s["v_cache"][at[0], g, at[1]].double()
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


def _exact_plan(s):
    """The tables one sequence, page and token at a time, in whole numbers on the host."""
    page, free, left = s["case"]["page"], s["free"].tolist(), int(s["n_free"][0])
    table, positions, slots = s["table"].tolist(), s["out"]["positions"].tolist(), s["out"]["slots"].tolist()
    q_start = [0]
    for row, c, n in zip(table, s["ctx"], s["new"]):
        for p in range(c, c + n):
            if p % page == 0:              # the first position of a page takes the last free one
                left -= 1
                row[p // page] = free[left]
            t = q_start[-1] + p - c
            positions[t], slots[t] = p, row[p // page] * page + p % page
        q_start.append(q_start[-1] + n)
    kv_len = [c + n for c, n in zip(s["ctx"], s["new"])]
    whole = {"table": table, "q_start": q_start, "kv_len": kv_len, "positions": positions, "slots": slots, "n_free": [left]}
    return {name: torch.tensor(x, dtype=torch.float64, device=GPU) for name, x in whole.items()}
