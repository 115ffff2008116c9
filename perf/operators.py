"""Measured cases of the paged-cache operators: writing new tokens into the packed FP8
cache, managing its pages, and attending from a chunk of new tokens over it.

A cache row is 584 bytes: 448 e4m3 values, 7 power-of-two scale bytes (one for 64
columns), a padding byte, 64 bf16 values.  The plain forms below state what each
operator computes in elementary torch operations."""
import math
import random

import torch

own = False

NOPE, ROPE, GROUP, ROW = 448, 64, 64, 584
SCALE = 1.0 / math.sqrt(512)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a serving batch writes one token a sequence
        {"name": "append_step_b96", "op": "append", "batch": 96, "n": 1, "ctx": 4001, "page": 64},
        # prompts of a prefill step, written at once
        {"name": "append_prompts_128k", "op": "append", "batch": 16, "n": 8192, "ctx": 8192, "page": 64},
        # a few branches of a sampling tree are dropped and forked again, and grow by a token
        {"name": "branch_n8", "op": "branch", "n": 8, "ctx": 2049, "page": 16, "pages": 8192, "grow": 1},
        # a large beam: every beam is dropped and forked from a survivor
        {"name": "branch_n512", "op": "branch", "n": 512, "ctx": 3000, "page": 64, "pages": 32768, "grow": 65},
        # a small pool after a few sequences ended
        {"name": "compact_1k_pages", "op": "compact", "pages": 1000, "page": 16, "used": 0.5, "rows": 16},
        # a large pool before its upper half is given back
        {"name": "compact_32k_pages", "op": "compact", "pages": 32768, "page": 64, "used": 0.4, "rows": 256},
        # verification of four drafted tokens: the latency case
        {"name": "verify_b4_n4_h64", "op": "chunk", "batch": 4, "n": 4, "heads": 64, "ctx": 1001, "page": 16,
         "cap": 0.0, "bias": False, "mask": "causal"},
        # a dense decode step: one token a sequence over its whole context
        {"name": "token_b32_h64_8k", "op": "chunk", "batch": 32, "n": 1, "heads": 64, "ctx": 8192, "page": 64,
         "cap": 0.0, "bias": False, "mask": "causal"},
        # one head shard of a long context
        {"name": "token_b2_h16_128k", "op": "chunk", "batch": 2, "n": 1, "heads": 16, "ctx": 131072, "page": 64,
         "cap": 0.0, "bias": False, "mask": "causal"},
        # a prefill chunk behind a cached context
        {"name": "chunk_n512_h64_8k", "op": "chunk", "batch": 1, "n": 512, "heads": 64, "ctx": 8192, "page": 64,
         "cap": 0.0, "bias": False, "mask": "causal"},
        # a mixed step of packed documents, capped scores and a distance bias; odd sizes and pages
        {"name": "mixed_b7_h16_capped", "op": "chunk", "batch": 7, "n": 301, "heads": 16, "ctx": 3001, "page": 48,
         "cap": 30.0, "bias": True, "mask": "documents"},
        # the largest prefill chunk, all heads on one GPU
        {"name": "chunk_n1024_h128_16k", "op": "chunk", "batch": 1, "n": 1024, "heads": 128, "ctx": 16384, "page": 64,
         "cap": 0.0, "bias": False, "mask": "causal"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "branch", "compact", "chunk", "chunk", "chunk"])
    page = rng.choice([1, 16, 48, 64, 64, 100])
    if op == "append":
        batch = _log(rng, 1, 96)
        n = _log(rng, 1, 131072 // batch)
        return {"op": op, "batch": batch, "n": n, "ctx": n + _log(rng, 1, 4096), "page": max(16, page)}
    if op == "branch":
        page, n = max(16, page), _log(rng, 1, 512)
        ctx, grow = _log(rng, 40, 2500), rng.choice([1, 4, 65])
        need = (n + 16) * ((ctx + grow) // page + 2)
        return {"op": op, "n": n, "ctx": ctx, "page": page, "pages": need + _log(rng, 100, 500000 // page), "grow": grow}
    if op == "compact":
        return {"op": op, "pages": _log(rng, 200, 32768), "page": max(16, min(page, 64)), "used": rng.uniform(0.1, 0.9),
                "rows": _log(rng, 8, 256)}
    while True:
        c = {"op": op, "batch": _log(rng, 1, 32), "n": _log(rng, 1, 1024), "heads": rng.choice([16, 32, 64, 128]),
             "page": page}
        c["ctx"] = max(c["n"], 1) + _log(rng, 1, 40000)
        rows = c["batch"] * c["n"] * c["heads"]
        if rows * c["ctx"] <= 1.2e9 and c["batch"] * c["ctx"] <= 300000:
            break
    c["cap"] = rng.choice([0.0, 0.0, 30.0, 50.0])
    c["bias"] = rng.random() < 0.3
    c["mask"] = rng.choice(["causal", "causal", "window", "documents", "prefix"])
    return c


def _lens(case):
    """Context lengths and new tokens of each sequence: around the case's, each its own."""
    r = random.Random("%s" % sorted((k, str(v)) for k, v in case.items() if k != "name"))
    B, n, ctx = case["batch"], case["n"], case["ctx"]
    if B == 1:
        return [ctx], [n]
    ns = [max(1, int(n * r.uniform(0.3, 1.0))) if case["op"] == "chunk" and n > 8 else n for _ in range(B)]
    ls = [max(m, int(ctx * r.uniform(0.5, 1.0))) if case["op"] == "append" or n > 1 else max(1, int(ctx * r.uniform(0.5, 1.5)))
          for m in ns]
    if case["op"] == "chunk" and case["ctx"] >= 100000:
        ls = [ctx] * B
    return ls, ns


def _visible(case, ls, ns):
    """(first, behind the last) visible position of every new token, or None for the causal mask."""
    if case["mask"] == "causal":
        return None
    lo, hi = [], []
    for L, n in zip(ls, ns):
        for j in range(n):
            p = L - n + j
            a, b = 0, p + 1
            if case["mask"] == "window":
                a = max(0, p - max(64, L // 4))
            elif case["mask"] == "documents":     # documents of about a third of the context
                d = max(1, L // 3)
                a = (p // d) * d
            elif case["mask"] == "prefix":        # the first half of the chunk sees itself whole
                b = max(b, L - n + n // 2)
            lo.append(a)
            hi.append(b)
    return lo, hi


def work(case):
    op, page = case["op"], case["page"]
    if op == "append":
        t = sum(_lens(case)[1])
        return {"bytes": t * (1024 + ROW) + 8 * case["batch"], "flops": t * 2 * NOPE}
    if op == "branch":
        ctx, n = case["ctx"], case["n"]
        rem, width = ctx % page, _width(case)
        return {"bytes": 2 * 4 * case["pages"] + 2 * n * rem * ROW + 5 * n * width * 4, "flops": 0}
    if op == "compact":
        used, rows, moved = _compact_counts(case)
        return {"bytes": 2 * moved * page * ROW + 2 * 4 * case["pages"] + 2 * 4 * used, "flops": 0}
    ls, ns = _lens(case)
    H, T = case["heads"], sum(ns)
    vis = _visible(case, ls, ns)
    if vis is None:
        pairs = sum(n * (L - n) + n * (n + 1) // 2 for L, n in zip(ls, ns))
        reach = sum(ls)
    else:
        pairs = sum(b - a for a, b in zip(*vis))
        reach, t = 0, 0
        for L, n in zip(ls, ns):
            reach += max(vis[1][t:t + n]) - min(vis[0][t:t + n])
            t += n
    return {"bytes": reach * ROW + T * H * (1024 + 896 + 4), "flops": 2.0 * H * 960 * pairs}


# ------------------------------------------------------------------ the packed rows
def _pack(x):
    """[n, 512] -> uint8 [n, 584]."""
    x = x.float()
    g = x[:, :NOPE].reshape(-1, 7, GROUP)
    amax = g.abs().amax(dim=2)
    m, e = torch.frexp(amax / 448.0)
    e = torch.where(m > 0.5, e, e - 1)
    byte = torch.where(amax == 0, torch.full_like(e, 127), (e + 127).clamp(1, 254))
    v = torch.ldexp(g, (127 - byte).unsqueeze(2)).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1, NOPE)
    pad = torch.zeros_like(byte[:, :1])
    rope = x[:, NOPE:].to(torch.bfloat16).view(torch.uint8).reshape(-1, 2 * ROPE)
    return torch.cat([v, byte.to(torch.uint8), pad.to(torch.uint8), rope], dim=1)


def _unpack(rows, dtype=torch.float32):
    """uint8 [n, 584] -> [n, 512]."""
    v = rows[:, :NOPE].contiguous().view(torch.float8_e4m3fn).to(dtype).view(-1, 7, GROUP)
    s = torch.ldexp(torch.ones((), dtype=dtype, device=rows.device), rows[:, NOPE:NOPE + 7].int() - 127)
    rope = rows[:, 456:ROW].contiguous().view(torch.bfloat16).to(dtype)
    return torch.cat([(v * s.unsqueeze(2)).view(-1, NOPE), rope], dim=1)


def _fill(pool, gen):
    for a in range(0, pool.shape[0], 1 << 18):
        b = min(pool.shape[0], a + (1 << 18))
        pool[a:b] = _pack(torch.randn(b - a, 512, generator=gen, device="cuda").to(torch.bfloat16))


def _width(case):
    return (case["ctx"] + case["grow"]) // case["page"] + 2


def _compact_counts(case):
    rows = case["rows"]
    per = max(1, int(case["pages"] * case["used"]) // rows)
    used = per * rows
    r = random.Random(case["pages"] * 31 + rows)
    at = sorted(r.sample(range(case["pages"]), used))
    return used, at, sum(p >= used for p in at)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    page, op = case["page"], case["op"]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    if op in ("append", "chunk"):
        ls, ns = _lens(case)
        width = max(-(-L // page) for L in ls) + 1
        count = sum(-(-L // page) for L in ls) + 7
        order = torch.randperm(count, generator=gen, device="cuda").int()
        table = torch.full((len(ls), width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, L in enumerate(ls):
            k = -(-L // page)
            table[b, :k] = order[at:at + k]
            at += k
        pool = torch.zeros(count * page, ROW, dtype=torch.uint8, device="cuda")
        T = sum(ns)
        s = {"op": op, "page": page, "pool": pool, "table": table, "kv_lens": ints(ls),
             "cu_q": ints([sum(ns[:b]) for b in range(len(ns) + 1)]), "most": max(ns), "longest": max(ls),
             "tokens": sum(ls), "batch": len(ls)}
        if op == "append":
            s["kv"] = (torch.randn(T, 512, generator=gen, device="cuda")
                       * torch.exp(torch.randn(T, 1, generator=gen, device="cuda"))).to(torch.bfloat16)
            return s
        _fill(pool, gen)
        H = case["heads"]
        s["q"] = torch.randn(T, H, 512, generator=gen, device="cuda").to(torch.bfloat16)
        s["cap"] = case["cap"]
        s["slopes"] = (torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H).float() if case["bias"] else None)
        vis = _visible(case, ls, ns)
        s["begin"], s["end"] = (None, None) if vis is None else (ints(vis[0]), ints(vis[1]))
        return s
    if op == "branch":
        n, ctx, width = case["n"], case["ctx"], _width(case)
        survivors = max(1, min(16, n // 4))
        R, k = survivors + n, -(-ctx // page)
        pages = case["pages"]
        order = torch.randperm(pages, generator=gen, device="cuda").int()
        table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
        table[:, :k] = order[:R * k].view(R, k)
        ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
        ref[order[:R * k].long()] = 1
        pool = torch.randint(0, 256, (pages * page, ROW), generator=gen, device="cuda", dtype=torch.uint8)
        lens = torch.full((R,), ctx, dtype=torch.int32, device="cuda")
        target = lens.clone()
        target[survivors:] += case["grow"]
        parents = torch.randint(0, survivors, (n,), generator=gen, device="cuda", dtype=torch.int32)
        children = survivors + torch.randperm(n, generator=gen, device="cuda").int()
        return {"op": op, "page": page, "pool": pool, "table": table, "ref": ref, "lens": lens, "parents": parents,
                "children": children, "target": target}
    used, at, _ = _compact_counts(case)
    rows, pages = case["rows"], case["pages"]
    ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
    ids = ints(at)
    ref[ids.long()] = 1
    table = ids[torch.randperm(used, generator=gen, device="cuda")].view(rows, used // rows).contiguous()
    pool = torch.randint(0, 256, (pages * page, ROW), generator=gen, device="cuda", dtype=torch.uint8)
    return {"op": op, "page": page, "pool": pool, "ref": ref, "table": table,
            "ref_out": torch.zeros_like(ref), "table_out": torch.zeros_like(table)}


# ------------------------------------------------------------------ the operators
def run(s):
    if own:
        import sparse_mla_decode_03_gb300 as m
    op, page, pool = s["op"], s["page"], s["pool"]
    if op == "append":
        if own:
            m.smla_cache_append(s["kv"], pool, s["table"], page, s["cu_q"], s["kv_lens"])
        else:
            rows = _rows_of(s)[_token_mask(s)]
            pool[rows] = _pack(s["kv"])
        return _held(pool)
    if op == "branch":
        if own:
            m.smla_cache_free(s["ref"], s["table"], s["lens"], s["children"])
            m.smla_cache_fork(pool, page, s["ref"], s["table"], s["lens"], s["parents"], s["children"])
            m.smla_cache_reserve(page, s["ref"], s["table"], s["target"])
        else:
            _free(s)
            _fork(s)
            _reserve(s)
        return {"pool": pool, "table": s["table"], "ref": s["ref"], "lens": s["lens"]}
    if op == "compact":
        if own:
            info = m.smla_cache_compact(pool, page, s["ref"], s["table"], ref_count_out=s["ref_out"],
                                        block_table_out=s["table_out"])
            return {"pool": pool, "table": s["table_out"], "ref": s["ref_out"], "info": info}
        return _compact(s)
    if own:
        out, lse = m.smla_chunk_attention(
            s["q"], pool, s["table"], page, s["cu_q"], s["kv_lens"], softmax_scale=SCALE, logit_cap=s["cap"],
            slopes=s["slopes"], vis_begin=s["begin"], vis_end=s["end"], max_kv_tokens=s["tokens"])
    else:
        out, lse = _chunk(s)
    return {"out": out, "lse": lse}


def _held(pool):
    return {"nope": pool[:, :NOPE].view(torch.float8_e4m3fn), "scales": pool[:, NOPE:456], "rope": pool[:, 456:].view(torch.bfloat16)}


def _token_mask(s):
    """[B, most]: which (sequence, new token) there are."""
    n = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    return torch.arange(s["most"], device="cuda").unsqueeze(0) < n.unsqueeze(1)


def _positions(s):
    n = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    return (s["kv_lens"].long() - n).unsqueeze(1) + torch.arange(s["most"], device="cuda").unsqueeze(0)


def _rows_of(s):
    """[B, most]: the pool row of every new token (any row where there is none)."""
    pos = _positions(s).clamp_min(0)
    cols = (pos // s["page"]).clamp_max(s["table"].shape[1] - 1)
    return s["table"].long().gather(1, cols) * s["page"] + pos % s["page"]


def _free(s):
    ref, table, rows = s["ref"], s["table"], s["children"].long()
    e = table[rows].reshape(-1).long()
    at = e.clamp_min(0)
    ref.index_add_(0, at, -(e >= 0).int())
    table[rows] = -1
    s["lens"][rows] = 0


def _take(ref, count):
    """The lowest free pages, at least `count` of them (page 0 again where there are too few)."""
    free = ref == 0
    rank = torch.cumsum(free.int(), 0) - 1
    ids = torch.zeros(ref.numel() + 1, dtype=torch.int64, device="cuda")
    ids[torch.where(free, rank.long(), ref.numel())] = torch.arange(ref.numel(), device="cuda")
    return ids[:count]


def _fork(s):
    ref, table, lens, page, pool = s["ref"], s["table"], s["lens"], s["page"], s["pool"]
    p, c = s["parents"].long(), s["children"].long()
    L = lens[p].long()
    full, rem = L // page, L % page
    col = torch.arange(table.shape[1], device="cuda").unsqueeze(0)
    src = table[p].long()
    shared = col < full.unsqueeze(1)
    part = rem > 0
    order = (torch.cumsum(part.int(), 0) - 1).clamp_min(0).long()
    fresh = _take(ref, p.numel())[order]
    last = src.gather(1, full.clamp_max(table.shape[1] - 1).unsqueeze(1)).squeeze(1)
    row = torch.arange(page, device="cuda").unsqueeze(0)
    sel = (row < rem.unsqueeze(1)).reshape(-1)
    pool[(fresh.unsqueeze(1) * page + row).reshape(-1)[sel]] = pool[(last.unsqueeze(1) * page + row).reshape(-1)[sel]]
    new = torch.where(shared, src, torch.full_like(src, -1))
    new = torch.where((col == full.unsqueeze(1)) & part.unsqueeze(1), fresh.unsqueeze(1), new)
    ref.index_add_(0, src.clamp_min(0).reshape(-1), shared.int().reshape(-1))
    ref.index_add_(0, fresh, part.int())
    table[c] = new.int()
    lens[c] = L.int()


def _reserve(s):
    ref, table, page = s["ref"], s["table"], s["page"]
    need = (s["target"].long() + page - 1) // page
    col = torch.arange(table.shape[1], device="cuda").unsqueeze(0)
    want = (col < need.unsqueeze(1)) & (table < 0)
    order = (torch.cumsum(want.reshape(-1).int(), 0) - 1).clamp_min(0).long()
    fresh = _take(ref, ref.numel())[order].view_as(table)
    table.copy_(torch.where(want, fresh.int(), table))
    ref.index_add_(0, fresh.reshape(-1), want.int().reshape(-1))


def _compact(s):
    pool, page, ref = s["pool"], s["page"], s["ref"]
    pages = ref.numel()
    ids = torch.arange(pages, device="cuda")
    used = ref > 0
    n_used = used.sum()
    hole = ~used & (ids < n_used)
    mover = used & (ids >= n_used)
    src, dst = ids[mover], ids[hole]
    pool.view(pages, page * ROW)[dst] = pool.view(pages, page * ROW)[src]
    to = ids.clone()
    to[src] = dst
    ref_out, table = s["ref_out"], s["table"]
    ref_out.copy_(ref)
    ref_out[dst] = ref[src]
    ref_out[src] = 0
    s["table_out"].copy_(torch.where(table >= 0, to[table.long().clamp_min(0)].int(), table))
    info = torch.stack([n_used, mover.sum()]).int()
    return {"pool": pool, "table": s["table_out"], "ref": ref_out, "info": info}


def _chunk(s):
    B, N, page, q = s["batch"], s["most"], s["page"], s["q"]
    H = q.shape[1]
    S = s["longest"]
    at = torch.arange(S, device="cuda")
    rows = s["table"].long()[:, at // page] * page + at % page
    kv = _unpack(s["pool"][rows.clamp_min(0).reshape(-1)]).view(B, S, 512)
    there = _token_mask(s)
    where = (s["cu_q"][:-1].long().unsqueeze(1) + torch.arange(N, device="cuda")).clamp_max(q.shape[0] - 1)
    x = torch.bmm(q[where].float().reshape(B, N * H, 512), kv.transpose(1, 2)).view(B, N, H, S).mul_(SCALE)
    if s["cap"]:
        x = x.div_(s["cap"]).tanh_().mul_(s["cap"])
    pos = _positions(s)
    if s["slopes"] is not None:
        away = (pos.unsqueeze(2) - at).abs().float()
        x -= s["slopes"].view(1, 1, H, 1) * away.unsqueeze(2)
    lo = torch.zeros_like(pos) if s["begin"] is None else s["begin"].long()[where]
    hi = pos + 1 if s["end"] is None else s["end"].long()[where]
    hi = torch.minimum(hi, s["kv_lens"].long().unsqueeze(1))
    seen = (at >= lo.unsqueeze(2)) & (at < hi.unsqueeze(2))
    x.masked_fill_(~seen.unsqueeze(2), float("-inf"))
    m = x.amax(dim=3, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    x = x.sub_(m).exp_()
    total = x.sum(dim=3, keepdim=True)
    o = torch.bmm(x.view(B, N * H, S), kv[:, :, :NOPE]).view(B, N, H, NOPE) / total.clamp_min(1e-38)
    lse = (m + total.log()).squeeze(3)
    return o[there].to(torch.bfloat16), lse[there]


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("branch", "compact"):
        return None
    ls, ns = _lens(case)
    page, pool, table = case["page"], s["pool"], s["table"].cpu().tolist()

    def rows(b, a, z):
        return torch.tensor([table[b][p // page] * page + p % page for p in range(a, z)], device="cuda")

    if op == "append":
        nope = torch.zeros(pool.shape[0], NOPE, dtype=torch.float64, device="cuda")
        rope = torch.zeros(pool.shape[0], ROPE, dtype=torch.float64, device="cuda")
        t = 0
        for b, (L, n) in enumerate(zip(ls, ns)):
            r, x = rows(b, L - n, L), s["kv"][t:t + n].double()
            t += n
            g = x[:, :NOPE].view(n, 7, GROUP)
            top = g.abs().amax(dim=2, keepdim=True)
            ratio = top / 448.0                  # the least e with 2^e >= ratio, counted up from below it
            e = torch.floor(torch.log2(ratio.clamp_min(2.0 ** -200))) - 1
            e = (e + sum((ratio > torch.exp2(e + k)).double() for k in range(3))).clamp(-126, 127)
            y = g / torch.exp2(torch.where(top == 0, torch.zeros_like(e), e))
            # e4m3 steps: 2^-9 below 2^-6, else an eighth of the power of two below
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
            nope[r] = (torch.round(y / step) * step).view(n, NOPE)
            rope[r] = x[:, NOPE:]
        return {"nope": nope, "scales": None, "rope": rope}
    out, lse, t = [], [], 0
    vis = _visible(case, ls, ns)
    H = case["heads"]
    for b, (L, n) in enumerate(zip(ls, ns)):
        kv = _unpack(pool[rows(b, 0, L)], torch.float64)
        at = torch.arange(L, device="cuda")
        pos = torch.arange(L - n, L, device="cuda")
        if vis is None:
            lo, hi = torch.zeros_like(pos), pos + 1
        else:
            lo, hi = (torch.tensor(v[t:t + n], device="cuda") for v in vis)
        seen = (at >= lo.unsqueeze(1)) & (at < hi.unsqueeze(1))
        away = (pos.unsqueeze(1) - at).abs().double()
        o = torch.empty(n, H, NOPE, dtype=torch.float64, device="cuda")
        z = torch.empty(n, H, dtype=torch.float64, device="cuda")
        for h in range(H):
            x = s["q"][t:t + n, h].double() @ kv.T * SCALE
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if s["slopes"] is not None:
                x = x - s["slopes"][h].double() * away
            x = x.masked_fill(~seen, float("-inf"))
            z[:, h] = torch.logsumexp(x, dim=1)
            o[:, h] = torch.exp(x - z[:, h:h + 1]) @ kv[:, :NOPE]
        out.append(o)
        lse.append(z)
        t += n
    return {"out": torch.cat(out), "lse": torch.cat(lse)}
