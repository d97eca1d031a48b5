"""Cases of the prompt side of the cache: page plans, per-head norms with the position rotation, attention of a chunk of
new tokens over the paged cache, and the tiers filled from the pages.

``own`` false: plain torch forms in 32 bits. ``own`` true: the calls of ``head_adaptive_kv_b200.prompt``."""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "fp32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
EPS = 1e-6
BASE = 1e6  # rotation base

# ---- cases ------------------------------------------------------------------
# plan: B requests, ctx tokens cached and new tokens joining (uniform in the ranges), `done` of the requests finished.
# norm: `tokens` rows of Hq + 2 Hkv heads. attn: B requests, ctx and new as for plan. fill: B requests of `ctx` tokens.


def listed():
    return [
        # one decode step of 64 requests: a page is needed only where a token crosses into it
        {"name": "plan_decode", "op": "plan", "B": 64, "page": 16, "ctx": "4096-32768", "new": "1-1", "done": 0, "lens": 11},
        # a step of a mixed server: prompts' chunks beside single tokens, a quarter of the requests finished and released
        {"name": "plan_mixed", "op": "plan", "B": 256, "page": 64, "ctx": "0-16384", "new": "1-127", "done": 64, "lens": 12},
        # the new token of 8 sequences on its way to the append: latency
        {"name": "norm_decode", "op": "norm", "tokens": 8, "Hq": 32, "Hkv": 8, "D": 128, "dtype": BF16, "page": 0, "rot": 128, "inter": False, "pos": 16384},
        # the chunk of a long prompt, K and V written to the pages
        {"name": "norm_prompt", "op": "norm", "tokens": 16384, "Hq": 32, "Hkv": 8, "D": 128, "dtype": BF16, "page": 64, "rot": 128, "inter": False, "pos": 65536},
        # 32-bit rows of the small fp32 workload's heads, half of each head rotated, odd count
        {"name": "norm_fp32", "op": "norm", "tokens": 999, "Hq": 4, "Hkv": 2, "D": 64, "dtype": F32, "page": 16, "rot": 32, "inter": True, "pos": 512},
        # one decode step over whole ragged contexts, before any tier is formed
        {"name": "attn_decode", "op": "attn", "B": 64, "Hq": 32, "Hkv": 8, "D": 128, "dtype": BF16, "page": 64, "ctx": "4096-32768", "new": "1-1", "lens": 21},
        # a few tokens behind a short context: the smallest call
        {"name": "attn_small_fp32", "op": "attn", "B": 1, "Hq": 4, "Hkv": 2, "D": 64, "dtype": F32, "page": 16, "ctx": "495-495", "new": "17-17", "lens": 22},
        # a mixed step: ragged chunks on ragged contexts
        {"name": "attn_mixed", "op": "attn", "B": 16, "Hq": 32, "Hkv": 8, "D": 128, "dtype": BF16, "page": 32, "ctx": "0-16384", "new": "1-1000", "lens": 23},
        # the second half of a 16k prompt
        {"name": "attn_prompt", "op": "attn", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "dtype": BF16, "page": 128, "ctx": "8192-8192", "new": "8192-8192", "lens": 24},
        # narrow heads, eight query heads to a KV head, small pages, odd lengths
        {"name": "attn_d64", "op": "attn", "B": 5, "Hq": 32, "Hkv": 4, "D": 64, "dtype": BF16, "page": 16, "ctx": "1-5000", "new": "333-1777", "lens": 25},
        # eight finished 16k prompts handed to the tiers
        {"name": "fill_16k", "op": "fill", "B": 8, "Hkv": 8, "D": 128, "dtype": BF16, "page": 64, "ctx": "15000-16320", "wcap": 256, "ncap": 16064, "lens": 31},
        # one short fp32 prompt
        {"name": "fill_fp32", "op": "fill", "B": 1, "Hkv": 2, "D": 64, "dtype": F32, "page": 16, "ctx": "496-496", "wcap": 64, "ncap": 432, "lens": 32},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _span(rng, lo, hi):
    a, b = sorted((_log(rng, lo, hi), _log(rng, lo, hi)))
    return "%d-%d" % (a, b)


def draw(rng):
    op = rng.choice(["plan", "norm", "attn", "attn", "attn", "fill"])
    page = rng.choice([16, 32, 64, 128, 256])
    lens = rng.randrange(1 << 30)
    dtype = rng.choice([BF16, BF16, BF16, F32])
    D = rng.choice([64, 128, 128])
    G, Hkv = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    if op == "plan":
        B = _log(rng, 1, 512)
        return {"op": op, "B": B, "page": page, "ctx": _span(rng, 1, 32768), "new": _span(rng, 1, max(1, 32768 // B)),
                "done": rng.choice([0, B // 4]), "lens": lens}
    if op == "norm":
        return {"op": op, "tokens": _log(rng, 1, 16384), "Hq": G * Hkv, "Hkv": Hkv, "D": D, "dtype": dtype, "page": rng.choice([0, page]),
                "rot": rng.choice([D, D, D // 2]), "inter": rng.random() < 0.3, "pos": _log(rng, 64, 131072)}
    if op == "fill":
        B = _log(rng, 1, 8)
        ctx = _span(rng, 16, 16320)
        return {"op": op, "B": B, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page, "ctx": ctx,
                "wcap": rng.choice([1, 64, 256, 500]), "ncap": _log(rng, 16, 16384), "lens": lens}
    while True:
        B = _log(rng, 1, 64)
        case = {"op": op, "B": B, "Hq": G * Hkv, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page, "ctx": _span(rng, 1, 32768),
                "new": "1-1" if rng.random() < 0.3 else _span(rng, 1, 8192), "lens": lens}
        w = work(case)
        if w["flops"] <= (1.6e12 if dtype == BF16 else 1e11) and w["bytes"] <= 5e9:
            return case
        lens += 1


def _lengths(case):
    """Each request's cached and new tokens: a function of the case alone."""
    r = random.Random(case["lens"])
    lo, hi = map(int, case["ctx"].split("-"))
    ctx = [r.randint(lo, hi) for _ in range(case["B"])]
    if "new" not in case:
        return ctx, [0] * case["B"]
    lo, hi = map(int, case["new"].split("-"))
    new = [r.randint(lo, hi) for _ in range(case["B"])]
    for b in range(case.get("done", 0)):
        new[b] = 0  # finished: these rows are released, and nothing joins them in this step
    return ctx, new


def _cdiv(a, b):
    return -(-a // b)


def work(case):
    op = case["op"]
    if op == "plan":
        ctx, new = _lengths(case)
        T, B, p = sum(new), case["B"], case["page"]
        pages = sum(_cdiv(c + n, p) - _cdiv(c, p) for c, n in zip(ctx, new))
        freed = sum(_cdiv(c, p) for c in ctx[:case["done"]])
        return {"bytes": 4.0 * (9 * B + 2 * T + 2 * pages + 2 * freed), "flops": float(B + T)}
    es = 2 if case["dtype"] == BF16 else 4
    if op == "norm":
        n = case["tokens"] * (case["Hq"] + 2 * case["Hkv"]) * case["D"]
        return {"bytes": 2.0 * n * es + 8.0 * case["tokens"], "flops": 8.0 * n}
    ctx, new = _lengths(case)
    if op == "fill":
        rows = sum(min(c, case["wcap"]) + min(max(0, c - case["wcap"]), case["ncap"]) for c in ctx)
        return {"bytes": 4.0 * rows * case["Hkv"] * case["D"] * es, "flops": 0.0}
    T, Hq, Hkv, D = sum(new), case["Hq"], case["Hkv"], case["D"]
    kv = sum(c + n for c, n in zip(ctx, new))
    seen = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    return {"bytes": 2.0 * T * Hq * D * es + 2.0 * kv * Hkv * D * es + 4.0 * T * Hq, "flops": 4.0 * D * Hq * seen}


# ---- inputs -----------------------------------------------------------------


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _randn(gen, shape, dtype):
    # drawn on the device in the type itself: caches of gigabytes are made quickly
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _table(r, lens, page, spare=0, cols=1):
    """Random pages for each request's tokens: (table rows of at least `cols` columns, pages in the pool, the pages nobody holds)."""
    held = [_cdiv(n, page) for n in lens]
    total = sum(held) + spare
    ids = list(range(total))
    r.shuffle(ids)
    cols = max(cols, max(held))
    rows, at = [], 0
    for h in held:
        rows.append(ids[at:at + h] + [-1] * (cols - h))
        at += h
    return rows, total, ids[at:]


def prepare(case, seed):
    r = random.Random(seed * 7 + 3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op == "plan":
        ctx, new = _lengths(case)
        page, B = case["page"], case["B"]
        need = sum(_cdiv(c + n, page) - _cdiv(c, page) for c, n in zip(ctx, new))
        held = [_cdiv(c, page) for c in ctx]
        rows, total, free = _table(r, ctx, page, need + 5, max(_cdiv(c + n, page) for c, n in zip(ctx, new)))
        T = sum(new) + 3  # a row capacity with a padded end
        s.update(ctx=_i32(ctx), new=_i32(new), held=_i32(held), table=_i32(rows), total=total,
                 free=_i32(free + [-1] * (total - len(free))), count=_i32([len(free)]),
                 done=_i32([1 if b < case["done"] else 0 for b in range(B)]), T=T,
                 held_out=_i32([0] * B), count_out=_i32([0]), granted=_i32([0] * B), q_start=_i32([0] * (B + 1)),
                 kv_len=_i32([0] * B), pos=_i32([0] * T), slot=_i32([0] * T))
        if own:
            from head_adaptive_kv_b200 import prompt
            s["state"] = prompt.PageState(s["table"], s["free"], s["count"], s["held"], page, total)
            s["after"] = prompt.PageState(s["table"], s["free"], s["count_out"], s["held_out"], page, total)
            s["chunk"] = prompt.Chunk(s["q_start"], s["kv_len"], s["pos"], s["slot"])
            s["ws"] = prompt.status_workspace("cuda")
        return s
    dt = DTYPES[case["dtype"]]
    if op == "norm":
        T, Hq, Hkv, D = case["tokens"], case["Hq"], case["Hkv"], case["D"]
        s["qkv"] = _randn(gen, (T, (Hq + 2 * Hkv) * D), dt) * 2
        s["qw"], s["kw"] = (1 + _randn(gen, (D,), dt) * 0.1 for _ in range(2))
        first = r.randrange(max(1, case["pos"] - T))
        s["pos"] = _i32(list(range(first, first + T)))
        half = case["rot"] // 2
        s["inv_freq"] = BASE ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        s["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device="cuda")
        if case["page"]:
            page = case["page"]
            slots = list(range(_cdiv(T, page) + 1))
            r.shuffle(slots)
            s["slot"] = _i32([slots[i // page] * page + i % page for i in range(T)])
            s["k"], s["v"] = (torch.zeros(len(slots), Hkv, page, D, dtype=dt, device="cuda") for _ in range(2))
        else:
            s["k"], s["v"] = (torch.zeros(T, Hkv, D, dtype=dt, device="cuda") for _ in range(2))
        if own:
            from head_adaptive_kv_b200 import hkv, prompt
            s["prob"] = hkv.Problem(1, Hq, Hkv, D, dt, 1.0, 0, 0)
            s["rope"] = prompt.Rope(s["inv_freq"], case["rot"], case["inter"])
            s["pages"] = prompt.Pages(s["k"], s["v"]) if case["page"] else None
            s["ws"] = prompt.status_workspace("cuda")
        return s
    ctx, new = _lengths(case)
    lens = [c + n for c, n in zip(ctx, new)]
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    rows, total, _ = _table(r, lens, page)
    s["k"], s["v"] = (_randn(gen, (total, Hkv, page, D), dt) for _ in range(2))
    s["table"], s["kv_len"], s["lens"] = _i32(rows), _i32(lens), lens
    if op == "fill":
        s["dk"], s["dv"] = (torch.zeros(B, Hkv, case["wcap"], D, dtype=dt, device="cuda") for _ in range(2))
        s["sk"], s["sv"] = (torch.zeros(B, Hkv, case["ncap"], D, dtype=dt, device="cuda") for _ in range(2))
        for name in ("dlen", "slen", "head", "dropped"):
            s[name] = _i32([0] * (B * Hkv))
        if own:
            from head_adaptive_kv_b200 import hkv, prompt
            s["prob"] = hkv.Problem(B, Hkv, Hkv, D, dt, 1.0, 0, 0)
            s["pages"] = prompt.Pages(s["k"], s["v"], s["table"])
            s["dense"], s["sparse"] = hkv.Tier(s["dk"], s["dv"], s["dlen"]), hkv.Tier(s["sk"], s["sv"], s["slen"])
            s["ws"] = prompt.status_workspace("cuda")
        return s
    Hq, T = case["Hq"], sum(new)
    s["new"] = new
    # queries of unit-norm-like heads: logits of a deviation near 1.5, as after the norms
    s["q"] = _randn(gen, (T, Hq, D), dt) * 1.5
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["q_start"], s["starts"] = _i32(starts), starts
    s["out"] = torch.zeros(T, Hq, D, dtype=dt, device="cuda")
    s["lse"] = torch.zeros(T, Hq, dtype=torch.float32, device="cuda")
    if own:
        from head_adaptive_kv_b200 import hkv, prompt
        s["prob"] = hkv.Problem(B, Hq, Hkv, D, dt, 1.0, 0, 0)
        s["pages"] = prompt.Pages(s["k"], s["v"], s["table"])
        s["ws"] = prompt.ChunkWorkspace(s["prob"], T, "cuda")
    return s


# ---- one pass ---------------------------------------------------------------


def run(s):
    return {"plan": _plan, "norm": _norm, "attn": _attn, "fill": _fill}[s["case"]["op"]](s)


def _plan(s):
    c = s["case"]
    if own:
        from head_adaptive_kv_b200 import prompt
        if c["done"]:
            prompt.page_release(s["done"], s["state"], s["after"], s["ws"])
            prompt.page_plan(s["ctx"], s["new"], s["after"], s["after"], s["chunk"], s["ws"], granted=s["granted"])
        else:
            prompt.page_plan(s["ctx"], s["new"], s["state"], s["after"], s["chunk"], s["ws"], granted=s["granted"])
        return _plan_out(s)
    page, T, table, free = c["page"], s["T"], s["table"], s["free"]
    ctx, new, held, count = s["ctx"].long(), s["new"].long(), s["held"].long(), s["count"].long()
    cols = torch.arange(table.shape[1], device="cuda")
    if c["done"]:
        back = torch.where(s["done"] != 0, held, 0)
        at = torch.cumsum(back, 0) - back
        where = count + at[:, None] + cols
        gone = cols < back[:, None]
        # pages that stay go to a place behind the list
        wide = torch.cat([free, free.new_zeros(1)])
        wide[torch.where(gone, where, free.numel()).reshape(-1)] = table.reshape(-1)
        free.copy_(wide[:-1])
        count = count + back.sum()
        held = held - back
    need = ((ctx + new + page - 1) // page - held).clamp(min=0)
    need = torch.where(new > 0, need, 0)
    ok = ((need == 0) | (torch.cumsum(need, 0) <= count)) & ((new == 0) | (torch.cumsum(new, 0) <= T))
    got, take = torch.where(ok, need, 0), torch.where(ok, new, 0)
    at = torch.cumsum(got, 0) - got
    fresh = (cols >= held[:, None]) & (cols < (held + got)[:, None])
    j = (count - 1 - (at[:, None] + cols - held[:, None])).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[j], table))
    ends = torch.cumsum(take, 0)
    s["q_start"][1:] = ends
    s["kv_len"].copy_(ctx + take)
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(ends, t, right=True)
    real = b < len(ends)
    b = b.clamp(max=len(ends) - 1)
    pos = ctx[b] + t - (ends - take)[b]
    col = (pos // page).clamp(0, table.shape[1] - 1)
    s["pos"].copy_(torch.where(real, pos, -1))
    s["slot"].copy_(torch.where(real, table[b, col].long() * page + pos % page, -1))
    s["granted"].copy_(take)
    s["held_out"].copy_(held + got)
    s["count_out"].copy_(count - got.sum())
    return _plan_out(s)


def _plan_out(s):
    return {k: s[k] for k in ("table", "free", "q_start", "kv_len", "pos", "slot", "granted", "held_out", "count_out")}


def _norm(s):
    c = s["case"]
    T, Hq, Hkv, D, rot, page = c["tokens"], c["Hq"], c["Hkv"], c["D"], c["rot"], c["page"]
    q, k, v = (x.unflatten(1, (-1, D)) for x in s["qkv"].split([Hq * D, Hkv * D, Hkv * D], 1))
    if own:
        from head_adaptive_kv_b200 import prompt
        if page:
            prompt.qk_norm_rope(s["prob"], q, k, v, s["pos"], s["rope"], s["q_out"], s["ws"], q_weight=s["qw"], k_weight=s["kw"],
                                eps=EPS, pages=s["pages"], slot=s["slot"])
        else:
            prompt.qk_norm_rope(s["prob"], q, k, v, s["pos"], s["rope"], s["q_out"], s["ws"], q_weight=s["qw"], k_weight=s["kw"],
                                eps=EPS, k_out=s["k"], v_out=s["v"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    angle = s["pos"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        head, rest = x[..., :rot], x[..., rot:]
        a, b = (head[..., 0::2], head[..., 1::2]) if c["inter"] else (head[..., :rot // 2], head[..., rot // 2:])
        a, b = a * cos - b * sin, b * cos + a * sin
        head = torch.stack([a, b], -1).flatten(-2) if c["inter"] else torch.cat([a, b], -1)
        return torch.cat([head, rest], -1).to(s["qkv"].dtype)

    s["q_out"].copy_(turned(q, s["qw"]))
    if page:
        slot = s["slot"].long()
        s["k"][slot // page, :, slot % page] = turned(k, s["kw"])
        s["v"][slot // page, :, slot % page] = v
    else:
        s["k"].copy_(turned(k, s["kw"]))
        s["v"].copy_(v)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _attn(s):
    c = s["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    if own:
        from head_adaptive_kv_b200 import prompt
        prompt.chunk_attention(s["prob"], s["q"], s["q_start"], s["kv_len"], s["pages"], s["out"], s["ws"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    G, scale = Hq // Hkv, D ** -0.5
    # requests one by one: padding them to the longest would multiply the work
    for b, n in enumerate(s["new"]):
        L, at = s["lens"][b], s["starts"][b]
        ids = s["table"][b, :_cdiv(L, page)]
        k, v = (x[ids].transpose(0, 1).reshape(Hkv, -1, D)[:, :L].float() for x in (s["k"], s["v"]))
        step = max(1, (1 << 29) // (Hq * L))  # rows at a time: 2 GB of scores
        for i in range(0, n, step):
            m = min(step, n - i)
            q = s["q"][at + i:at + i + m].float().view(m, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * m, D)
            score = (q @ k.transpose(1, 2)).mul_(scale).view(Hkv, G, m, L)
            if n > 1:
                last = L - n + i + torch.arange(m, device="cuda")[:, None]
                score.masked_fill_(torch.arange(L, device="cuda") > last, -math.inf)
            top = score.amax(-1, keepdim=True)
            p = score.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            o = (p.view(Hkv, G * m, L) @ v).view(Hkv, G, m, D) / total
            s["out"][at + i:at + i + m] = o.permute(2, 0, 1, 3).reshape(m, Hq, D).to(s["out"].dtype)
            s["lse"][at + i:at + i + m] = (top + total.log())[..., 0].permute(2, 0, 1).reshape(m, Hq)
    return {"out": s["out"], "lse": s["lse"]}


def _fill(s):
    c = s["case"]
    B, Hkv, page, W, n = c["B"], c["Hkv"], c["page"], c["wcap"], c["ncap"]
    if own:
        from head_adaptive_kv_b200 import prompt
        prompt.fill_tiers(s["prob"], s["pages"], s["kv_len"], s["dense"], s["head"], s["sparse"], s["ws"], dropped=s["dropped"])
        return _fill_out(s)
    L = s["kv_len"].long()
    slot = torch.arange(W, device="cuda")
    oldest = (L - W).clamp(min=0)[:, None]
    in_window = oldest + (slot - oldest) % W
    row = torch.arange(n, device="cuda").expand(B, n)
    for t, real, k, v in ((in_window, in_window < L[:, None], s["dk"], s["dv"]), (row, row < (L - W)[:, None], s["sk"], s["sv"])):
        t = torch.where(real, t, 0)
        ids = torch.gather(s["table"].long(), 1, t // page)
        for src, dst in ((s["k"], k), (s["v"], v)):
            dst.copy_(torch.where(real[:, None, :, None], src[ids, :, t % page].transpose(1, 2), dst))
    per_unit = lambda x: x.to(torch.int32).repeat_interleave(Hkv)  # noqa: E731
    aged = (L - W).clamp(min=0)
    s["dlen"].copy_(per_unit(L.clamp(max=W)))
    s["head"].copy_(per_unit(torch.where(L > W, L % W, 0)))
    s["slen"].copy_(per_unit(aged.clamp(max=n)))
    s["dropped"].copy_(per_unit((aged - n).clamp(min=0)))
    return _fill_out(s)


def _fill_out(s):
    return {k: s[k] for k in ("dk", "dv", "dlen", "head", "sk", "sv", "slen", "dropped")}


# ---- 64 bits ----------------------------------------------------------------


def exact(case, seed):
    """The operators' definitions in 64 bits. Page plans and fills have no computed numbers."""
    op = case["op"]
    if op in ("plan", "fill"):
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    D = case["D"]
    if op == "norm":
        Hq, Hkv, rot = case["Hq"], case["Hkv"], case["rot"]
        x = s["qkv"].double().view(case["tokens"], Hq + 2 * Hkv, D)
        w = torch.cat([s["qw"].double().expand(Hq, D), s["kw"].double().expand(Hkv, D)])
        y = x[:, :Hq + Hkv]
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + EPS) * w
        i = torch.arange(rot // 2, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["inter"] else (i, i + rot // 2)
        z = torch.view_as_complex(torch.stack([y[..., first], y[..., second]], -1))
        z = z * torch.exp(1j * (s["pos"].double()[:, None] * s["inv_freq"]))[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        k, v = y[:, Hq:], x[:, Hq + Hkv:]
        if case["page"]:
            slot = s["slot"].long()
            flat = [torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
            for f, rows in zip(flat, (k, v)):
                f[slot // case["page"], :, slot % case["page"]] = rows
            k, v = flat
        return {"q": y[:, :Hq].contiguous(), "k": k.contiguous(), "v": v.contiguous()}
    Hq, Hkv, page = case["Hq"], case["Hkv"], case["page"]
    G = Hq // Hkv
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["new"]):
        L, at = s["lens"][b], s["starts"][b]
        j = torch.arange(L, device="cuda")
        ids = s["table"][b].long()[j // page]
        step = max(1, (1 << 27) // L)
        for h in range(Hkv):
            k, v = s["k"][ids, h, j % page].double(), s["v"][ids, h, j % page].double()
            for g in range(h * G, h * G + G):
                for i in range(0, n, step):
                    rows = torch.arange(i, min(n, i + step), device="cuda")
                    a = s["q"][at + rows, g].double() @ k.T / math.sqrt(D)
                    a = torch.where(j <= (L - n + rows)[:, None], a, -math.inf)
                    z = torch.logsumexp(a, 1)
                    out[at + rows, g] = torch.exp(a - z[:, None]) @ v
                    lse[at + rows, g] = z
    return {"out": out, "lse": lse}
