"""Measured cases of the operators around a beam-searched decode step: appending tokens to the
paged cache with the position rotation applied on the way, the cache in 4-bit rows (written,
read back, attended to densely and through a list of positions), the selection over beams and
vocabulary, and the reordering of the cache by the selected parents.

A 4-bit row is 368 bytes: 224 of e2m1 values (a word of 4 bytes holds columns 8 i .. 8 i + 7,
column 2 p of them in nibble p and column 2 p + 1 in nibble p + 4), 14 power-of-two scale bytes
(one for 32 columns), 2 of padding, 64 bf16 values.  An 8-bit row is 584 bytes: 448 e4m3 values,
7 power-of-two scale bytes (one for 64 columns), a padding byte, 64 bf16 values.  The plain forms
below state what each operator computes in elementary torch operations."""
import math
import random

import torch

own = False

NOPE, ROPE = 448, 64
ROW8, ROW4 = 584, 368
SCALE = 1.0 / math.sqrt(512)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
NIBBLE_OF = (0, 4, 1, 5, 2, 6, 3, 7)          # of column 8 i + k in word i


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a serving batch: a token a sequence is written, its queries rotated
        {"name": "rotary_step_b96_h64", "op": "rotary", "rows": 8, "batch": 96, "n": 1, "ctx": 4001, "page": 64,
         "heads": 64, "pairs": "interleaved"},
        # prompts of a prefill step, one shard of the heads
        {"name": "rotary_prompts_64k_h16", "op": "rotary", "rows": 8, "batch": 16, "n": 4096, "ctx": 4096, "page": 64,
         "heads": 16, "pairs": "interleaved"},
        # prompts written to 4-bit rows and read back as the attention sees them; odd lengths and pages
        {"name": "rotary_4bit_b5_n2001", "op": "rotary", "rows": 4, "batch": 5, "n": 2001, "ctx": 2500, "page": 48,
         "heads": 16, "pairs": "halves"},
        # sparse decode step of a serving batch over flat 4-bit rows
        {"name": "sparse4_b32_h64_k2048", "op": "sparse", "batch": 32, "heads": 64, "topk": 2048, "ctx": 16384, "page": 0},
        # the same over pages, a shard of the heads, an odd number of positions
        {"name": "sparse4_paged_b96_h16_k999", "op": "sparse", "batch": 96, "heads": 16, "topk": 999, "ctx": 8000, "page": 64},
        # verification of four drafted tokens over 4-bit rows: the latency case
        {"name": "verify4_b4_n4_h64", "op": "chunk", "batch": 4, "n": 4, "heads": 64, "ctx": 1001, "page": 16, "mask": "causal"},
        # a dense decode step over 4-bit rows
        {"name": "token4_b32_h64_8k", "op": "chunk", "batch": 32, "n": 1, "heads": 64, "ctx": 8192, "page": 64, "mask": "causal"},
        # the largest: a prefill chunk of all heads behind a cached context, in a sliding window
        {"name": "chunk4_n512_h128_12k", "op": "chunk", "batch": 1, "n": 512, "heads": 128, "ctx": 12345, "page": 64,
         "mask": "window"},
        # one request with four beams
        {"name": "select_g1_k4_32k", "op": "select", "groups": 1, "beams": 4, "out": 4, "vocab": 32000, "type": "float32",
         "done": False},
        # a batch of requests with eight beams each, twice as many candidates kept, some beams finished
        {"name": "select_g64_k8_128k", "op": "select", "groups": 64, "beams": 8, "out": 16, "vocab": 131072,
         "type": "bfloat16", "done": True},
        # every beam of a batch goes on from a survivor of its group
        {"name": "reorder_g2_k4", "op": "reorder", "rows": 8, "groups": 2, "beams": 4, "ctx": 2049, "page": 16, "pages": 8192},
        {"name": "reorder_g64_k8", "op": "reorder", "rows": 4, "groups": 64, "beams": 8, "ctx": 3000, "page": 64, "pages": 32768},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "sparse", "chunk", "chunk", "select", "reorder"])
    page = rng.choice([1, 16, 48, 64, 64, 100])
    if op == "rotary":
        batch = _log(rng, 1, 96)
        n = _log(rng, 1, 65536 // batch)
        rows = rng.choice([4, 8])
        return {"op": op, "rows": rows, "batch": batch, "n": min(n, 20000 // batch + 1) if rows == 4 else n,
                "ctx": n + _log(rng, 1, 4096), "page": max(16, page), "heads": rng.choice([1, 12, 16]),
                "pairs": rng.choice(["interleaved", "halves"])}
    if op == "sparse":
        batch = _log(rng, 1, 96)
        return {"op": op, "batch": batch, "heads": rng.choice([16, 32, 64, 128]), "topk": _log(rng, 1, min(8192, 131072 // batch)),
                "ctx": _log(rng, 1, 16384), "page": rng.choice([0, page])}
    if op == "select":
        groups, beams = _log(rng, 1, 64), rng.randint(1, 12)
        out = rng.choice([beams, 2 * beams])
        return {"op": op, "groups": groups, "beams": beams, "out": out, "vocab": _log(rng, 50, 67000000 // max(512, groups * beams)),
                "type": rng.choice(["float32", "bfloat16", "float16"]), "done": rng.random() < 0.4}
    if op == "reorder":
        groups, beams, page = _log(rng, 1, 64), rng.randint(1, 8), max(16, page)
        ctx = _log(rng, 1, 2500)
        need = groups * beams * (ctx // page + 3)
        return {"op": op, "rows": rng.choice([4, 8]), "groups": groups, "beams": beams, "ctx": ctx, "page": page,
                "pages": need + _log(rng, 100, 500000 // page)}
    while True:
        c = {"op": op, "batch": _log(rng, 1, 32), "n": _log(rng, 1, 512), "heads": rng.choice([16, 32, 64, 128]),
             "page": page}
        c["ctx"] = max(c["n"], 1) + _log(rng, 1, 30000)
        if c["batch"] * c["n"] * c["heads"] * c["ctx"] <= 8e8 and c["batch"] * c["ctx"] <= 250000:
            break
    c["mask"] = rng.choice(["causal", "causal", "window", "documents", "prefix"])
    return c


def _lens(case):
    """Context lengths and new tokens of each sequence: around the case's, each its own."""
    r = random.Random("%s" % sorted((k, str(v)) for k, v in case.items() if k != "name"))
    B, n, ctx = case["batch"], case.get("n", 1), case["ctx"]
    if B == 1:
        return [ctx], [n]
    ns = [max(1, int(n * r.uniform(0.3, 1.0))) if case["op"] == "chunk" and n > 8 else n for _ in range(B)]
    return [max(m, int(ctx * r.uniform(0.5, 1.0)) + 1) for m in ns], ns


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
                a = max(0, p - max(64, 3 * L // 4))
            elif case["mask"] == "documents":     # documents of about a third of the context
                d = max(1, L // 3)
                a = (p // d) * d
            elif case["mask"] == "prefix":        # the first half of the chunk sees itself whole
                b = max(b, L - n + n // 2)
            lo.append(a)
            hi.append(b)
    return lo, hi


def _row_bytes(case):
    return ROW8 if case.get("rows") == 8 else ROW4


def work(case):
    op, row = case["op"], _row_bytes(case)
    if op == "rotary":
        ls, ns = _lens(case)
        T, H = sum(ns), case["heads"]
        table = 4 * ROPE * max(ls)
        back = 1024 * T if case["rows"] == 4 else 0
        return {"bytes": T * (1024 + row + 256 * H) + min(table, 4 * ROPE * T) + back, "flops": T * (2 * NOPE + 3 * ROPE * (H + 1))}
    if op == "sparse":
        B, H, k = case["batch"], case["heads"], case["topk"]
        return {"bytes": B * k * (row + 4) + B * H * (1024 + 896 + 4), "flops": 2.0 * H * 960 * B * k}
    if op == "select":
        rows = case["groups"] * case["beams"]
        read = rows - (sum(_finished(case)) if case["done"] else 0)
        size = 4 if case["type"] == "float32" else 2
        return {"bytes": read * case["vocab"] * size + rows * 5 + case["groups"] * case["out"] * 12,
                "flops": 3.0 * read * case["vocab"]}
    if op == "reorder":
        R, ctx, page = case["groups"] * case["beams"], case["ctx"], case["page"]
        extra = R - len(set(_parents(case)))
        return {"bytes": 4 * case["pages"] + 2 * extra * (ctx % page) * row + 3 * 4 * R * (ctx // page + 1), "flops": 0}
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
    return {"bytes": reach * row + T * H * (1024 + 896 + 4), "flops": 2.0 * H * 960 * pairs}


def _parents(case):
    """Which row each beam goes on from: within its group, about half of the beams survive."""
    r = random.Random(case["groups"] * 977 + case["beams"] * 31 + case["ctx"])
    K, got = case["beams"], []
    for g in range(case["groups"]):
        kept = r.sample(range(K), (K + 1) // 2)
        got += [g * K + r.choice(kept) for _ in range(K)]
    return got


def _finished(case):
    r = random.Random(case["groups"] * 131 + case["beams"])
    return [r.random() < 0.1 for _ in range(case["groups"] * case["beams"])]


# ------------------------------------------------------------------ the packed rows
def _pack8(x, rope):
    """x [n, 448], rope bf16 [n, 64] -> uint8 [n, 584]."""
    g = x.float().reshape(-1, 7, 64)
    amax = g.abs().amax(dim=2)
    m, e = torch.frexp(amax / 448.0)
    e = torch.where(m > 0.5, e, e - 1)
    byte = torch.where(amax == 0, torch.full_like(e, 127), (e + 127).clamp(1, 254))
    v = torch.ldexp(g, (127 - byte).unsqueeze(2)).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1, NOPE)
    pad = torch.zeros_like(byte[:, :1])
    return torch.cat([v, byte.to(torch.uint8), pad.to(torch.uint8), rope.contiguous().view(torch.uint8).reshape(-1, 128)], dim=1)


def _pack4(x, rope):
    """x [n, 448], rope bf16 [n, 64] -> uint8 [n, 368]."""
    g = x.float().reshape(-1, 14, 32)
    amax = g.abs().amax(dim=2)
    m, e = torch.frexp(amax / 6.0)
    e = torch.where(m > 0.5, e, e - 1)
    byte = torch.where(amax == 0, torch.full_like(e, 127), (e + 127).clamp(1, 254))
    y = torch.ldexp(g, (127 - byte).unsqueeze(2))
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() + (a >= 3.5).int()
            + (a > 5.0).int() + 8 * torch.signbit(y).int()).reshape(-1, 56, 8)
    nib = torch.empty_like(code)
    nib[:, :, list(NIBBLE_OF)] = code
    v = (nib[:, :, 0::2] + 16 * nib[:, :, 1::2]).to(torch.uint8).reshape(-1, 224)
    pad = torch.zeros(byte.shape[0], 2, dtype=torch.uint8, device=x.device)
    return torch.cat([v, byte.to(torch.uint8), pad, rope.contiguous().view(torch.uint8).reshape(-1, 128)], dim=1)


def _unpack4(rows, dtype=torch.float32):
    """uint8 [n, 368] -> [n, 512]."""
    b = rows[:, :224].int()
    nib = torch.stack([b & 15, b >> 4], dim=2).view(-1, 56, 8)[:, :, list(NIBBLE_OF)].reshape(-1, 14, 32)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=rows.device)
    s = torch.ldexp(torch.ones((), dtype=dtype, device=rows.device), rows[:, 224:238].int() - 127)
    rope = rows[:, 240:ROW4].contiguous().view(torch.bfloat16).to(dtype)
    return torch.cat([(table[nib.long()] * s.unsqueeze(2)).reshape(-1, NOPE), rope], dim=1)


def _fill4(pool, gen):
    for a in range(0, pool.shape[0], 1 << 17):
        b = min(pool.shape[0], a + (1 << 17))
        x = torch.randn(b - a, 512, generator=gen, device="cuda").to(torch.bfloat16)
        pool[a:b] = _pack4(x[:, :NOPE], x[:, NOPE:])


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if op == "select":
        G, K, V = case["groups"], case["beams"], case["vocab"]
        # logits of a model that is sure of itself now and then: scaled normal values
        x = normal(G * K, V) * (1.5 + torch.rand(G * K, 1, generator=gen, device="cuda") * 1.5)
        s = {"op": op, "logits": x.to(getattr(torch, case["type"])), "scores": -20.0 * torch.rand(G, K, generator=gen, device="cuda"),
             "out": case["out"], "end": 2 % V,
             "done": torch.tensor(_finished(case), device="cuda").to(torch.uint8) if case["done"] else None}
        return s
    if op == "reorder":
        page, ctx, pages, row = case["page"], case["ctx"], case["pages"], _row_bytes(case)
        R, k = case["groups"] * case["beams"], -(-ctx // page)
        width = ctx // page + 2
        order = torch.randperm(pages, generator=gen, device="cuda").int()
        table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
        table[:, :k] = order[:R * k].view(R, k)
        ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
        ref[order[:R * k].long()] = 1
        pool = torch.randint(0, 256, (pages * page, row), generator=gen, device="cuda", dtype=torch.uint8)
        return {"op": op, "page": page, "pool": pool, "table": table, "ref": ref, "parents": ints(_parents(case)),
                "lens": torch.full((R,), ctx, dtype=torch.int32, device="cuda")}
    page = case["page"] or case["ctx"]
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
    pool = torch.zeros(count * page, _row_bytes(case), dtype=torch.uint8, device="cuda")
    T, H = sum(ns), case["heads"]
    s = {"op": op, "page": page, "pool": pool, "table": table, "kv_lens": ints(ls), "batch": len(ls), "tokens": sum(ls),
         "cu_q": ints([sum(ns[:b]) for b in range(len(ns) + 1)]), "most": max(ns), "longest": max(ls)}
    if op == "rotary":
        s["kv"] = (normal(T, 512) * torch.exp(normal(T, 1))).to(torch.bfloat16)
        s["q_rope"] = normal(T, H, ROPE).to(torch.bfloat16)
        s["q"] = torch.zeros(T, H, 512, dtype=torch.bfloat16, device="cuda")
        s["interleaved"], s["bits"] = case["pairs"] == "interleaved", case["rows"]
        angle = (torch.arange(max(ls), dtype=torch.float64, device="cuda").unsqueeze(1)
                 * torch.pow(10000.0, -torch.arange(32, dtype=torch.float64, device="cuda") / 32))
        s["rotary"] = torch.cat([torch.cos(angle), torch.sin(angle)], dim=1).float()
        return s
    _fill4(pool, gen)
    if op == "sparse":
        B, k = case["batch"], case["topk"]
        s["q"] = normal(B, H, 512).to(torch.bfloat16)
        pos = (torch.rand(B, k, generator=gen, device="cuda") * s["kv_lens"].unsqueeze(1)).long()
        masked = torch.rand(B, k, generator=gen, device="cuda") < 0.02
        if case["page"]:
            idx = pos
        else:                       # rows of the pool
            s["paged"] = False
            idx = s["table"].long().gather(1, pos // page) * page + pos % page
        s["paged"] = bool(case["page"])
        s["indices"] = torch.where(masked, -1, idx).int()
        return s
    s["q"] = normal(T, H, 512).to(torch.bfloat16)
    vis = _visible(case, ls, ns)
    s["begin"], s["end"] = (None, None) if vis is None else (ints(vis[0]), ints(vis[1]))
    return s


# ------------------------------------------------------------------ the operators
def run(s):
    if own:
        import sparse_mla_decode_03_gb300 as m
    op = s["op"]
    if op == "select":
        if own:
            parents, tokens, scores = m.smla_beam_select(s["logits"], s["scores"], num_out=s["out"], finished=s["done"],
                                                         end_token=s["end"])
        else:
            parents, tokens, scores = _select(s)
        return {"parents": parents, "tokens": tokens, "scores": scores}
    if op == "reorder":
        if own:
            m.smla_cache_reorder(s["pool"], s["page"], s["ref"], s["table"], s["lens"], s["parents"])
        else:
            _reorder(s)
        return {"pool": s["pool"], "table": s["table"], "ref": s["ref"], "lens": s["lens"]}
    page, pool = s["page"], s["pool"]
    if op == "rotary":
        if own:
            m.smla_cache_append_rotary(s["kv"], pool, s["table"], page, s["cu_q"], s["kv_lens"], s["rotary"],
                                       interleaved=s["interleaved"], q_rope=s["q_rope"], q=s["q"])
        else:
            _append(s)
        if s["bits"] == 8:
            return {"q": s["q"], "nope": pool[:, :NOPE].view(torch.float8_e4m3fn), "scales": pool[:, NOPE:456],
                    "rope": pool[:, 456:].view(torch.bfloat16)}
        if own:
            back = m.smla_cache_read(pool, s["table"], page, s["cu_q"], s["kv_lens"], s["kv"].shape[0])
        else:
            back = _unpack4(pool[_rows_of(s)[_token_mask(s)]]).to(torch.bfloat16)
        return {"q": s["q"], "kv": back}
    if op == "sparse":
        if not own:
            out, lse = _sparse(s)
        elif s["paged"]:
            out, lse = m.sparse_mla_decode_paged(s["q"], pool, s["table"], page, s["indices"], SCALE)
        else:
            out, lse = m.sparse_mla_decode(s["q"], pool, s["indices"], SCALE)
    elif own:
        out, lse = m.smla_chunk_attention(s["q"], pool, s["table"], page, s["cu_q"], s["kv_lens"], softmax_scale=SCALE,
                                          vis_begin=s["begin"], vis_end=s["end"], max_kv_tokens=s["tokens"])
    else:
        out, lse = _chunk(s)
    return {"out": out, "lse": lse}


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


def _rotate(x, turn, interleaved):
    """x [..., 64] bf16, turn [..., 64] (cosines of the 32 pairs, then sines)."""
    x, c, d = x.float(), turn[..., :32], turn[..., 32:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * d, a * d + b * c], dim=-1).flatten(-2).to(torch.bfloat16)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * c - b * d, a * d + b * c], dim=-1).to(torch.bfloat16)


def _append(s):
    there = _token_mask(s)
    turn = s["rotary"][_positions(s)[there]]
    kv = s["kv"]
    pack = _pack8 if s["bits"] == 8 else _pack4
    s["pool"][_rows_of(s)[there]] = pack(kv[:, :NOPE], _rotate(kv[:, NOPE:], turn, s["interleaved"]))
    s["q"][:, :, NOPE:] = _rotate(s["q_rope"], turn.unsqueeze(1), s["interleaved"])


def _select(s):
    x = s["logits"].double()                     # the order of near scores counts
    G, K = s["scores"].shape
    V, n = x.shape[1], s["out"]
    top = x.amax(dim=1, keepdim=True)
    x = x - (top + (x - top).exp().sum(dim=1, keepdim=True).log())
    if s["done"] is not None:
        only = torch.full((V,), float("-inf"), dtype=torch.float64, device="cuda")
        only[s["end"]] = 0.0
        x = torch.where(s["done"].bool().unsqueeze(1), only, x)
    x = (x + s["scores"].double().view(-1, 1)).view(G, K * V)
    v, at = torch.sort(x, dim=1, descending=True, stable=True)     # equal ones: the lowest first
    n_there = min(n, K * V)
    v, at = v[:, :n_there], at[:, :n_there]
    none = v == float("-inf")
    base = torch.arange(G, device="cuda").unsqueeze(1) * K
    parents = torch.where(none, -1, base + at // V).int()
    tokens = torch.where(none, -1, at % V).int()
    more = n - n_there
    pad = torch.nn.functional.pad
    return pad(parents, (0, more), value=-1), pad(tokens, (0, more), value=-1), pad(v.float(), (0, more), value=float("-inf"))


def _reorder(s):
    ref, table, lens, page, pool = s["ref"], s["table"], s["lens"], s["page"], s["pool"]
    R, p = table.shape[0], s["parents"].long()
    r = torch.arange(R, device="cuda")
    col = torch.arange(table.shape[1], device="cuda").unsqueeze(0)
    first = torch.full_like(r, R).scatter_reduce(0, p, r, "amin")      # the child that takes a row over
    dropped = (first == R).unsqueeze(1) & (table >= 0)
    ref.index_add_(0, table.clamp_min(0).reshape(-1).long(), -dropped.reshape(-1).int())
    L, src = lens[p].long(), table[p].long()
    full, rem = L // page, L % page
    more = first[p] != r                         # the others share full pages and copy a last one
    part = more & (rem > 0)
    shared = more.unsqueeze(1) & (col < full.unsqueeze(1))
    free = ref == 0
    rank = torch.cumsum(free.int(), 0) - 1
    ids = torch.zeros(ref.numel() + 1, dtype=torch.int64, device="cuda")
    ids[torch.where(free, rank.long(), ref.numel())] = torch.arange(ref.numel(), device="cuda")
    fresh = ids[(torch.cumsum(part.int(), 0) - 1).clamp_min(0).long()]
    last = src.gather(1, full.clamp_max(table.shape[1] - 1).unsqueeze(1)).squeeze(1)
    row = torch.arange(page, device="cuda").unsqueeze(0)
    sel = ((row < rem.unsqueeze(1)) & part.unsqueeze(1)).reshape(-1)
    pool[(fresh.unsqueeze(1) * page + row).reshape(-1)[sel]] = pool[(last.unsqueeze(1) * page + row).reshape(-1)[sel]]
    ref.index_add_(0, src.clamp_min(0).reshape(-1), shared.reshape(-1).int())
    ref.index_add_(0, fresh, part.int())
    new = torch.where(more.unsqueeze(1) & ~shared, -1, src)
    new = torch.where(part.unsqueeze(1) & (col == full.unsqueeze(1)), fresh.unsqueeze(1), new)
    table.copy_(new.int())
    lens.copy_(L.int())


def _attend(q, kv, seen):
    """q [B, M, 512], kv [B, S, 512] fp32, seen [B, M or 1, S] -> out bf16 [B, M, 448], lse [B, M]."""
    x = torch.bmm(q.float(), kv.transpose(1, 2)).mul_(SCALE)
    x.masked_fill_(~seen, float("-inf"))
    m = x.amax(dim=2, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    x = x.sub_(m).exp_()
    total = x.sum(dim=2, keepdim=True)
    o = torch.bmm(x, kv[:, :, :NOPE]) / total.clamp_min(1e-38)
    return o.to(torch.bfloat16), (m + total.log()).squeeze(2)


def _sparse(s):
    idx = s["indices"].long()
    rows = idx.clamp_min(0)
    if s["paged"]:
        rows = s["table"].long().gather(1, rows // s["page"]) * s["page"] + rows % s["page"]
    kv = _unpack4(s["pool"][rows.reshape(-1)]).view(*idx.shape, 512)
    return _attend(s["q"], kv, (idx >= 0).unsqueeze(1))


def _chunk(s):
    B, N, page, q = s["batch"], s["most"], s["page"], s["q"]
    H, S = q.shape[1], s["longest"]
    at = torch.arange(S, device="cuda")
    rows = s["table"].long()[:, at // page] * page + at % page
    kv = _unpack4(s["pool"][rows.clamp_min(0).reshape(-1)]).view(B, S, 512)
    there = _token_mask(s)
    where = (s["cu_q"][:-1].long().unsqueeze(1) + torch.arange(N, device="cuda")).clamp_max(q.shape[0] - 1)
    pos = _positions(s)
    lo = torch.zeros_like(pos) if s["begin"] is None else s["begin"].long()[where]
    hi = pos + 1 if s["end"] is None else s["end"].long()[where]
    hi = torch.minimum(hi, s["kv_lens"].long().unsqueeze(1))
    seen = (at >= lo.unsqueeze(2)) & (at < hi.unsqueeze(2))
    seen = seen.unsqueeze(2).expand(B, N, H, S).reshape(B, N * H, S)
    out, lse = _attend(q[where].reshape(B, N * H, 512), kv, seen)
    return out.view(B, N, H, NOPE)[there], lse.view(B, N, H)[there]


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    op = case["op"]
    if op == "reorder":
        return None
    s = prepare(case, seed)
    if op == "select":
        return _exact_select(case, s)
    ls, ns = _lens(case)
    page, pool, table = s["page"], s["pool"], s["table"].cpu().tolist()

    def rows(b, a, z):
        return torch.tensor([table[b][p // page] * page + p % page for p in range(a, z)], device="cuda")

    if op == "rotary":
        kv, q_rope, turn = s["kv"].double(), s["q_rope"].double(), s["rotary"].double()
        # a pair as a complex number, turned by another
        pos = torch.cat([torch.arange(L - n, L, device="cuda") for L, n in zip(ls, ns)])
        z = torch.complex(turn[pos, :32], turn[pos, 32:])

        def turned(x, by):
            w = torch.view_as_complex(x.unflatten(-1, (32, 2)).contiguous()) if s["interleaved"] else torch.complex(x[..., :32], x[..., 32:])
            w = w * by
            return torch.view_as_real(w).flatten(-2) if s["interleaved"] else torch.cat([w.real, w.imag], dim=-1)

        q = torch.zeros(*q_rope.shape[:2], 512, dtype=torch.float64, device="cuda")
        q[:, :, NOPE:] = turned(q_rope, z.unsqueeze(1))
        k_rope = turned(kv[:, NOPE:], z)
        width, grid_max, least = (64, 448.0, 2.0 ** -6) if case["rows"] == 8 else (32, 6.0, 1.0)
        bits = 3 if case["rows"] == 8 else 1
        g = kv[:, :NOPE].reshape(kv.shape[0], -1, width)
        top = g.abs().amax(dim=2, keepdim=True)
        ratio = top / grid_max               # the least e with 2^e >= ratio, counted up from below it
        e = torch.floor(torch.log2(ratio.clamp_min(2.0 ** -200))) - 1
        e = (e + sum((ratio > torch.exp2(e + k)).double() for k in range(3))).clamp(-126, 127)
        e = torch.where(top == 0, torch.zeros_like(e), e)
        y = g / torch.exp2(e)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(least))) - bits)
        held = torch.round(y / step) * step      # in units of the scale
        if case["rows"] == 4:
            return {"q": q, "kv": torch.cat([(held * torch.exp2(e)).reshape(-1, NOPE), k_rope], dim=1)}
        nope = torch.zeros(pool.shape[0], NOPE, dtype=torch.float64, device="cuda")
        rope = torch.zeros(pool.shape[0], ROPE, dtype=torch.float64, device="cuda")
        at = torch.cat([rows(b, L - n, L) for b, (L, n) in enumerate(zip(ls, ns))])
        nope[at], rope[at] = held.reshape(-1, NOPE), k_rope
        return {"q": q, "nope": nope, "scales": None, "rope": rope}
    H = case["heads"]
    out, lse, t = [], [], 0
    if op == "sparse":
        idx = s["indices"].cpu().tolist()
        for b in range(case["batch"]):
            at = [i for i in idx[b] if i >= 0]
            if s["paged"]:
                at = [table[b][i // page] * page + i % page for i in at]
            kv = _held4(pool[torch.tensor(at, dtype=torch.int64, device="cuda")])
            x = s["q"][b].double() @ kv.T * SCALE
            z = torch.logsumexp(x, dim=1)
            out.append(torch.exp(x - z[:, None]) @ kv[:, :NOPE])
            lse.append(z)
        z = torch.stack(lse)
        return {"out": torch.nan_to_num(torch.stack(out)), "lse": z}
    vis = _visible(case, ls, ns)
    for b, (L, n) in enumerate(zip(ls, ns)):
        kv = _held4(pool[rows(b, 0, L)])
        at, pos = torch.arange(L, device="cuda"), torch.arange(L - n, L, device="cuda")
        if vis is None:
            lo, hi = torch.zeros_like(pos), pos + 1
        else:
            lo, hi = (torch.tensor(v[t:t + n], device="cuda") for v in vis)
        seen = (at >= lo.unsqueeze(1)) & (at < hi.unsqueeze(1))
        o = torch.empty(n, H, NOPE, dtype=torch.float64, device="cuda")
        z = torch.empty(n, H, dtype=torch.float64, device="cuda")
        for h in range(H):
            x = (s["q"][t:t + n, h].double() @ kv.T * SCALE).masked_fill(~seen, float("-inf"))
            z[:, h] = torch.logsumexp(x, dim=1)
            o[:, h] = torch.exp(x - z[:, h:h + 1]) @ kv[:, :NOPE]
        out.append(o)
        lse.append(z)
        t += n
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


def _held4(rows):
    """uint8 [n, 368] -> the 64-bit values that they stand for, a bit field at a time."""
    word = rows[:, :224].contiguous().view(torch.int32).long() & 0xffffffff
    v = torch.empty(rows.shape[0], 56, 8, dtype=torch.float64, device=rows.device)
    for k in range(8):
        f = (word >> (4 * (k // 2 + 4 * (k % 2)))) & 15
        ex, man = (f >> 1) & 3, (f & 1).double()
        mag = torch.where(ex == 0, 0.5 * man, (1 + 0.5 * man) * torch.exp2((ex - 1).double()))
        v[:, :, k] = torch.where(f >= 8, -mag, mag)
    v = v.view(-1, 14, 32) * torch.exp2(rows[:, 224:238].double() - 127).unsqueeze(2)
    return torch.cat([v.view(-1, NOPE), rows[:, 240:ROW4].contiguous().view(torch.bfloat16).double()], dim=1)


def _exact_select(case, s):
    G, K, V, n = case["groups"], case["beams"], case["vocab"], case["out"]
    done = s["done"].cpu().tolist() if s["done"] is not None else [0] * (G * K)
    parents, tokens, scores = [], [], []
    for g in range(G):
        found = []
        for k in range(K):
            r, base = g * K + k, float(s["scores"][g, k])
            if done[r]:
                found.append((-base, r, s["end"]))
                continue
            x = torch.log_softmax(s["logits"][r].double(), dim=0)
            least = torch.topk(x, min(n, V)).values[-1]
            at = (x >= least).nonzero().squeeze(1)
            found += [(-(base + v), r, i) for v, i in zip(x[at].tolist(), at.tolist())]
        found = sorted(found)[:n]
        found += [(float("inf"), -1, -1)] * (n - len(found))
        parents.append([f[1] for f in found])
        tokens.append([f[2] for f in found])
        scores.append([-f[0] for f in found])
    return {"parents": torch.tensor(parents, dtype=torch.int32), "tokens": torch.tensor(tokens, dtype=torch.int32),
            "scores": torch.tensor(scores, dtype=torch.float64)}
