"""Chunk attention over the paged cache against the definition in 64 bits, and the run of the
cache calls and the attention together.  Tolerances are derived in _cache_helpers."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_03_gb300 as m

from _cache_helpers import (ROW, SCALE, check_chunk, chunk_reference, dev, pack_rows, random_pool, tables)

pytestmark = pytest.mark.gpu


def _case(lens, ns, H, page, seed, stride=ROW, lead=0, mult=1.0, extra=1):
    num_pages = sum(-(-max(L, 0) // page) for L in lens) + 2
    pool = random_pool(num_pages, page, seed, stride, lead, mult)
    table = tables(lens, page, num_pages, seed, extra)
    cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((max(1, int(cu[-1])), H, 512), generator=g).to(torch.bfloat16).cuda()
    return q, pool, table, cu, np.array(lens, np.int32)


def _run(q, pool, table, page, cu, lens, cap=0.0, slopes=None, begin=None, end=None, status=0, **kw):
    m.smla_device_status(clear=True)
    got = m.smla_chunk_attention(q, pool, dev(table), page, dev(cu), dev(lens), softmax_scale=SCALE, logit_cap=cap,
                                 slopes=slopes, vis_begin=None if begin is None else dev(begin),
                                 vis_end=None if end is None else dev(end), **kw)
    assert m.smla_device_status(clear=True) == status
    return got


def _check(q, pool, table, page, cu, lens, cap=0.0, slopes=None, begin=None, end=None, **kw):
    got = _run(q, pool, table, page, cu, lens, cap, slopes, begin, end, **kw)
    check_chunk(got, chunk_reference(q, pool, table, page, cu, lens, SCALE, cap, slopes, begin, end))
    return got


SHAPES = [
    # lens, new tokens, H, page
    ([1], [1], 64, 1),
    ([1, 2, 3], [1, 1, 3], 16, 1),
    ([64, 63, 65, 0, 1], [1, 1, 1, 0, 1], 64, 16),
    ([1001, 700, 30], [4, 1, 4], 64, 16),
    ([300, 5000], [1, 1], 32, 48),
    ([257], [3], 128, 64),
    ([130, 128, 127], [2, 1, 3], 128, 33),
    ([700, 450], [200, 37], 16, 100),
    ([65], [65], 64, 64),
    ([513, 80], [130, 80], 32, 64),
    ([400], [140], 128, 7),
    ([2500, 0, 1300, 90], [64, 0, 33, 90], 64, 64),
]


@pytest.mark.parametrize("lens,ns,H,page", SHAPES)
def test_causal(lens, ns, H, page):
    _check(*_pick(_case(lens, ns, H, page, seed=H + page + len(lens)), page))


def _pick(c, page):
    q, pool, table, cu, lens = c
    return q, pool, table, page, cu, lens


def _masks(kind, lens, ns, seed):
    rng = np.random.default_rng(seed)
    begin, end = [], []
    for L, n in zip(lens, ns):
        for j in range(n):
            p = L - n + j
            a, b = 0, p + 1
            if kind == "window":
                a = p - 70
            elif kind == "documents":
                a = p // 100 * 100
            elif kind == "prefix":
                b = max(b, L - n // 2)
            elif kind == "random":         # anything goes: empty, negative, past the end, one token
                a, b = (int(v) for v in rng.integers(-20, L + 40, 2))
            elif kind == "empty":
                a, b = (5, 5) if j % 3 else (L, L + 9)
            begin.append(a)
            end.append(b)
    return np.array(begin, np.int32), np.array(end, np.int32)


@pytest.mark.parametrize("kind", ["window", "documents", "prefix", "random", "empty"])
@pytest.mark.parametrize("lens,ns,H,page", [([900, 333], [40, 70], 64, 48), ([600, 77, 1], [1, 1, 1], 64, 16),
                                            ([500], [300], 16, 64), ([260, 300], [64, 9], 128, 100)])
def test_masks(kind, lens, ns, H, page):
    c = _case(lens, ns, H, page, seed=3 * H + len(kind))
    begin, end = _masks(kind, lens, ns, seed=H)
    _check(*_pick(c, page), begin=begin, end=end)


@pytest.mark.parametrize("which", ["begin", "end"])
def test_one_sided_masks(which):
    lens, ns, page = [300, 280], [20, 130], 64
    c = _case(lens, ns, 64, page, seed=5)
    begin, end = _masks("window" if which == "begin" else "prefix", lens, ns, 5)
    _check(*_pick(c, page), begin=begin if which == "begin" else None, end=end if which == "end" else None)


@pytest.mark.parametrize("cap,bias", [(30.0, False), (0.0, True), (5.0, True), (0.01, False)])
@pytest.mark.parametrize("lens,ns,H,page", [([1200, 40], [1, 1], 64, 64), ([700, 300], [150, 64], 16, 48),
                                            ([300], [70], 128, 64)])
def test_cap_and_distance_bias(cap, bias, lens, ns, H, page):
    c = _case(lens, ns, H, page, seed=int(H + 10 * cap))
    slopes = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H).float() if bias else None
    begin, end = _masks("prefix", lens, ns, 1)
    _check(*_pick(c, page), cap=cap, slopes=slopes, begin=begin, end=end)


@pytest.mark.parametrize("n,H", [(1, 64), (130, 64), (90, 16)])
def test_scores_that_rise_along_the_context(n, H):
    """The running maximum grows by far more than any headroom from block to block, again and
    again, and falls at the end."""
    L, page = 700, 64
    q, pool, table, cu, lens = _case([L], [n], H, page, seed=9)
    q = q.abs()
    x = torch.rand(L, 512, generator=torch.Generator().manual_seed(1)) * torch.linspace(0.0, 12.0, L)[:, None]
    x[-90:] *= 0.05
    rows = dev(pack_rows(x.to(torch.bfloat16)))
    at = torch.as_tensor(table[0].astype(np.int64)[np.arange(L) // page] * page + np.arange(L) % page, device="cuda")
    pool[at] = rows
    _check(q, pool, table, page, cu, lens)


def test_large_values_and_unusual_scales():
    """Rows beyond the f16 range, tiny rows and extreme scale bytes keep their values."""
    L, page, H = 200, 16, 64
    for n in (1, 140):
        q, pool, table, cu, lens = _case([L], [n], H, page, seed=21)
        q = (q.float() * 2.0 ** -9).to(torch.bfloat16)
        g = torch.Generator().manual_seed(2)
        x = torch.randn(L, 512, generator=g)
        x[::7, :64] *= 2.0 ** 14
        x[3::7, 64:128] *= 2.0 ** -40
        x[5::7, 200:300] = 0
        at = torch.as_tensor(table[0].astype(np.int64)[np.arange(L) // page] * page + np.arange(L) % page,
                             device="cuda")
        pool[at] = dev(pack_rows(x.to(torch.bfloat16)))
        _check(q, pool, table, page, cu, lens)


@pytest.mark.parametrize("n,H", [(1, 64), (2, 16), (150, 64)])
def test_unmapped_pages_and_pages_past_the_pool(n, H):
    L, page = 520, 16
    q, pool, table, cu, lens = _case([L, 300], [n, n], H, page, seed=31)
    table[0, 3] = table[0, 11] = -1
    table[1, 0] = -7
    _check(q, pool, table, page, cu, lens)
    table[0, 20] = pool.shape[0] // page            # the first page id past the pool
    table[1, 5] = 2 ** 31 - 1
    _check(q, pool, table, page, cu, lens, status=-7)
    table[:, :] = -1
    _check(q, pool, table, page, cu, lens)          # nothing is mapped


@pytest.mark.parametrize("n", [1, 150])
def test_lengths_past_the_table(n):
    L, page, H = 130, 16, 64
    q, pool, table, cu, lens = _case([L], [n if n < L else L - 1], H, page, seed=33, extra=0)
    cut = table[:, :6].copy()
    _check(q, pool, cut, page, cu, lens, status=-7)


@pytest.mark.parametrize("n", [3, 200])
def test_more_new_tokens_than_the_length(n):
    q, pool, table, cu, lens = _case([n // 2 + 1, 40], [n, 5], 64, 16, seed=35)
    _check(q, pool, table, 16, cu, lens)


@pytest.mark.parametrize("n", [2, 140])
def test_entries_outside_every_sequence_are_left_alone(n):
    H, page = 64, 64
    q, pool, table, cu, lens = _case([300, 200], [n, n], H, page, seed=37)
    q = torch.cat([q, q[:9]]).contiguous()
    cu = cu + 4
    out = torch.full((q.shape[0], H, 448), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], H), 7.0, device="cuda")
    got = _check(q, pool, table, page, cu, lens, out=out, lse=lse)
    for t in list(range(4)) + list(range(4 + 2 * n, q.shape[0])):
        assert (got[0][t] == 7).all() and (got[1][t] == 7).all()


@pytest.mark.parametrize("stride,lead", [(592, 16), (600, 0), (1024, 32)])
@pytest.mark.parametrize("n", [1, 135])
def test_strided_pools(stride, lead, n):
    q, pool, table, cu, lens = _case([333], [n], 64, 48, seed=41, stride=stride, lead=lead)
    _check(q, pool, table, 48, cu, lens)


def test_large_ragged_batch():
    rng = np.random.default_rng(7)
    lens = [int(v) for v in rng.integers(0, 900, 70)]
    ns = [int(min(L, v)) for L, v in zip(lens, rng.integers(0, 9, 70))]
    _check(*_pick(_case(lens, ns, 16, 32, seed=43), 32))


def test_a_bound_on_the_tokens_that_is_exact_or_too_small():
    lens, ns, page = [700, 260], [140, 70], 64
    c = _case(lens, ns, 64, page, seed=45)
    a = _run(*_pick(c, page), max_kv_tokens=sum(lens))
    b = _run(*_pick(c, page))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_same_call_twice_gives_the_same_bits():
    for ns in ([1, 1], [150, 90]):
        c = _case([3000, 700], ns, 64, 64, seed=47)
        a, b = _run(*_pick(c, 64)), _run(*_pick(c, 64))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("ns", [[1, 1], [130, 70]])
def test_graph_replay_follows_new_lengths_and_side_streams(ns):
    page, H = 64, 64
    q, pool, table, cu, lens = _case([800, 700], ns, H, page, seed=51)
    t, c, l = dev(table), dev(cu), dev(lens)
    p = m.make_chunk_params(2, H, q.shape[0], page, table.shape[1], pool.shape[0], ROW, 1500)
    ws = torch.empty(m.smla_chunk_workspace_size(p), dtype=torch.uint8, device="cuda")
    out = torch.empty((q.shape[0], H, 448), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((q.shape[0], H), device="cuda")
    s = torch.cuda.Stream()

    def call():
        m.smla_chunk_attention(q, pool, t, page, c, l, softmax_scale=SCALE, max_kv_tokens=1500, out=out, lse=lse,
                               workspace=ws, stream=s)

    s.wait_stream(torch.cuda.current_stream())
    call()
    s.synchronize()
    check_chunk((out, lse), chunk_reference(q, pool, table, page, cu, lens))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for new in ([800, 700], [401, 130], [140, 650]):
        l.copy_(dev(np.array(new, np.int32)))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        check_chunk((out, lse), chunk_reference(q, pool, table, page, cu, np.array(new, np.int32)))


def test_two_calls_at_once_on_two_streams():
    cases = [_case([1500, 600], [1, 3], 64, 64, seed=61), _case([900], [140], 32, 48, seed=62)]
    pages = [64, 48]
    want = [_run(*_pick(c, p)) for c, p in zip(cases, pages)]
    streams = [torch.cuda.Stream() for _ in cases]
    args = [(q, pool, dev(t), p, dev(cu), dev(l)) for (q, pool, t, cu, l), p in zip(cases, pages)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for a, s in zip(args, streams):
            with torch.cuda.stream(s):
                got.append(m.smla_chunk_attention(*a, softmax_scale=SCALE))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_single_tokens_agree_with_the_sparse_decode_over_all_positions():
    """A chunk of one token a sequence is the decode step with every position selected."""
    lens, page, H = [500, 129, 64], 64, 64
    q, pool, table, cu, l = _case(lens, [1, 1, 1], H, page, seed=71)
    out, lse = _run(q, pool, table, page, cu, l)
    idx = np.full((3, 500), -1, np.int32)
    for b, L in enumerate(lens):
        idx[b, :L] = np.arange(L)
    o2, z2 = m.sparse_mla_decode_paged(q, pool, dev(table), page, dev(idx), softmax_scale=SCALE)
    assert (out.float() - o2.float()).abs().max() <= 1e-2        # the decode path's own bar
    assert (lse - z2).abs().max() <= 1e-3


def test_cache_calls_and_attention_together():
    """A serving loop: prompts are reserved, written and attended, a sequence is forked, the
    branches grow apart, one is dropped, the pool is compacted, and the rest goes on; every
    step's attention is checked against rows packed from the tokens themselves."""
    page, num_pages, R, width, H = 16, 80, 4, 20, 64
    gen = torch.Generator().manual_seed(5)
    pool = torch.full((num_pages * page, ROW), 0x11, dtype=torch.uint8, device="cuda")
    ref = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    tokens = [torch.zeros(0, 512, dtype=torch.bfloat16) for _ in range(R)]

    def step(ns):
        cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        kv = torch.randn(int(cu[-1]), 512, generator=gen).to(torch.bfloat16)
        q = torch.randn(int(cu[-1]), H, 512, generator=gen).to(torch.bfloat16).cuda()
        for r, n in enumerate(ns):
            tokens[r] = torch.cat([tokens[r], kv[cu[r]:cu[r] + n]])
        lens.add_(dev(np.array(ns, np.int32)))
        m.smla_cache_reserve(page, ref, table, lens)
        m.smla_cache_append(kv.cuda(), pool, table, page, dev(cu), lens)
        got = m.smla_chunk_attention(q, pool, table, page, dev(cu), lens, softmax_scale=SCALE)
        # the oracle reads rows packed from the tokens, one after another, not the pool
        L = [t.shape[0] for t in tokens]
        flat = torch.cat([dev(pack_rows(t)) for t in tokens if t.shape[0]] + [torch.zeros(1, ROW, dtype=torch.uint8,
                                                                                         device="cuda")])
        at = np.full((R, max(L)), -1, np.int32)
        for r in range(R):
            at[r, :L[r]] = sum(L[:r]) + np.arange(L[r])
        assert lens.cpu().tolist() == L
        check_chunk(got, chunk_reference(q, flat, at, 1, cu, np.array(L, np.int32)))

    m.smla_device_status(clear=True)
    step([70, 33, 0, 0])
    step([1, 1, 0, 0])
    m.smla_cache_fork(pool, page, ref, table, lens, dev(np.array([0, 0], np.int32)), dev(np.array([2, 3], np.int32)))
    tokens[2], tokens[3] = tokens[0].clone(), tokens[0].clone()
    step([0, 1, 4, 1])
    m.smla_cache_free(ref, table, lens, dev(np.array([1], np.int32)))
    tokens[1] = tokens[1][:0]
    info = m.smla_cache_compact(pool, page, ref, table)
    used = int((ref > 0).sum())
    assert info.cpu().tolist()[0] == used and bool((ref[:used] > 0).all())
    step([1, 20, 1, 130])
    assert m.smla_device_status(clear=True) == 0


def test_binding_refusals():
    q, pool, table, cu, lens = _case([50], [3], 64, 16, seed=81)
    t, c, l = dev(table), dev(cu), dev(lens)
    bad = [
        lambda: m.smla_chunk_attention(q.float(), pool, t, 16, c, l),
        lambda: m.smla_chunk_attention(q[:, :, :500], pool, t, 16, c, l),
        lambda: m.smla_chunk_attention(q, pool, t.long(), 16, c, l),
        lambda: m.smla_chunk_attention(q, pool, t, 16, c[:1], l),
        lambda: m.smla_chunk_attention(q, pool, t, 16, c, l.cpu()),
        lambda: m.smla_chunk_attention(q, pool, t, 0, c, l),
        lambda: m.smla_chunk_attention(q, pool, t, 16, c, l, slopes=torch.ones(32, device="cuda")),
        lambda: m.smla_chunk_attention(q, pool, t, 16, c, l, vis_begin=l),
        lambda: m.smla_chunk_attention(q, pool, t, 16, c, l, out=torch.empty(3, 64, 448, device="cuda")),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for kw in ({"softmax_scale": -1.0}, {"logit_cap": -2.0}, {"max_kv_tokens": 0},
               {"workspace": torch.empty(1, dtype=torch.uint8, device="cuda")}):
        with pytest.raises(m.SmlaError):
            m.smla_chunk_attention(q, pool, t, 16, c, l, **kw)
    with pytest.raises(m.SmlaError):
        m.smla_chunk_attention(q[:, :48].contiguous(), pool, t, 16, c, l)


@pytest.mark.parametrize("n,H", [(1, 64), (3, 16), (70, 64), (150, 16)])
def test_rows_that_are_not_finite_reach_only_who_sees_them(n, H):
    """NaN and infinities in the cache: a token that sees such a row gets NaN, every other is
    what it is without it (masked, causal later or in a page's unused tail)."""
    L, page = 300, 48
    q, pool, table, cu, lens = _case([L], [n], H, page, seed=91)
    row = lambda p: int(table[0, p // page]) * page + p % page      # noqa: E731
    pool[row(40), 7] = 0x7F                       # e4m3 NaN
    pool[row(41), 450] = 0xFF                     # a NaN scale
    pool[row(42), 449] = 250                      # a scale past bf16
    pool[row(130), 500:502] = torch.tensor([0x80, 0x7F], dtype=torch.uint8)      # an infinite rope value
    tail = int(table[0, -2]) * page + page - 1    # behind the last token of the last page
    pool[tail] = 0xFF
    begin = np.array([(0, 43, 131, 200)[j % 4] for j in range(n)], np.int32)
    end = np.array([L - n + j + 1 if j % 3 else 35 for j in range(n)], np.int32)
    out, lse = _run(q, pool, table, page, cu, lens, begin=begin, end=end)
    clean = pool.clone()
    for p in (40, 41, 42, 130):
        clean[row(p)] = 0
    ref = chunk_reference(q, clean, table, page, cu, lens, begin=begin, end=end)
    sees = torch.tensor([any(b <= p < e for p in (40, 41, 42, 130)) for b, e in zip(begin, end)], device="cuda")
    assert torch.isnan(out[sees].float()).all() and torch.isnan(lse[sees]).all()
    ref[0][sees] = ref[1][sees] = float("nan")    # (not compared)
    check_chunk((out, lse), ref)


@pytest.mark.parametrize("n,H", [(2, 64), (100, 64)])
def test_query_rows_that_are_not_finite_stay_alone(n, H):
    q, pool, table, cu, lens = _case([200], [n], H, 64, seed=93)
    ref = chunk_reference(q, pool, table, 64, cu, lens)
    q[1, 5, 100] = float("nan")
    q[0, 3, 500] = float("inf")
    out, lse = _run(q, pool, table, 64, cu, lens)
    for t, h in ((1, 5), (0, 3)):
        assert torch.isnan(out[t, h].float()).all() and torch.isnan(lse[t, h])
        out[t, h], lse[t, h] = ref[0][t, h].to(torch.bfloat16), ref[1][t, h].float()
    check_chunk((out, lse), ref)


@pytest.mark.parametrize("n", [1, 140])
def test_tokens_past_the_bound_are_masked_and_reported(n):
    """max_kv_tokens too small: the first sequences keep their tokens, later ones what is left,
    counted in blocks of 64 with one to spare for every sequence."""
    lens, page = [320, 640, 256], 64
    q, pool, table, cu, l = _case(lens, [n] * 3, 64, page, seed=95)
    got = _run(q, pool, table, page, cu, l, max_kv_tokens=448, status=-7)       # 7 + 3 blocks: 5, 5, 0
    cut = table.copy()
    cut[1, 5:] = -1
    cut[2] = -1
    check_chunk(got, chunk_reference(q, pool, cut, page, cu, l))


@pytest.mark.parametrize("n,H", [(1, 16), (17, 16)])
def test_more_sequences_than_the_plan_keeps_on_chip(n, H):
    rng = np.random.default_rng(3)
    lens = [int(v) for v in rng.integers(0, 70, 2100)]
    ns = [min(L, int(v)) for L, v in zip(lens, rng.integers(0, n + 1, 2100))]
    lens[5] = 300
    q, pool, table, cu, l = _case(lens, ns, H, 16, seed=97)
    out, lse = _run(q, pool, table, 16, cu, l)
    pick = [0, 5, 1023, 1024, 1025, 2047, 2048, 2099] + [int(v) for v in rng.integers(0, 2100, 60)]
    for b in pick:                                  # each against the definition by itself
        if ns[b] == 0:
            continue
        rows = slice(int(cu[b]), int(cu[b + 1]))
        ref = chunk_reference(q[rows], pool, table[b:b + 1], 16, [0, ns[b]], [lens[b]])
        check_chunk((out[rows], lse[rows]), ref)


@pytest.mark.parametrize("n", [1, 130])
def test_a_pool_past_four_gigabytes(n):
    """Row offsets past 32 bits: the pages in use are the last of the pool."""
    page, H, L = 64, 64, 500
    num_pages = (1 << 32) // (ROW * page) + 70
    pool = torch.zeros(num_pages * page, ROW, dtype=torch.uint8, device="cuda")
    small = random_pool(10, page, 99)
    pool[-10 * page:] = small
    table = (num_pages - 10 + np.random.default_rng(1).permutation(10)[None, :9]).astype(np.int32)
    lens = np.array([L], np.int32)
    cu = np.array([0, n], np.int32)
    q = torch.randn(n, H, 512, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    kv = torch.randn(n, 512, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    m.smla_cache_append(kv.cuda(), pool, dev(table), page, dev(cu), dev(lens))
    assert (pool[:-10 * page].view(-1)[::4097] == 0).all()
    got = _run(q, pool, table, page, cu, lens)
    low = table - (num_pages - 10)
    check_chunk(got, chunk_reference(q, pool[-10 * page:], low, page, cu, lens))
    at = torch.as_tensor(low[0].astype(np.int64)[np.arange(L - n, L) // page] * page + np.arange(L - n, L) % page)
    assert np.array_equal(pool[-10 * page:].cpu().numpy()[at.numpy()], pack_rows(kv))


def test_single_row_pools_and_single_positions():
    """One page of one row, one token: the smallest cache there is."""
    q, pool, table, cu, lens = _case([1], [1], 128, 1, seed=101)
    one = pool[int(table[0, 0]):int(table[0, 0]) + 1]
    _check(q, one, np.zeros((1, 1), np.int32), 1, cu, lens)


def test_no_sequence_has_new_tokens():
    q, pool, table, cu, lens = _case([50, 20], [0, 0], 64, 16, seed=103)
    out = torch.full((1, 64, 448), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, 64), 3.0, device="cuda")
    _run(q, pool, table, 16, cu, lens, out=out, lse=lse)
    assert (out == 3).all() and (lse == 3).all()


@pytest.mark.parametrize("ns", [[1, 1], [140, 60]])
def test_calls_that_follow_one_another_share_a_workspace(ns):
    """Calls of different shapes in one stream, one workspace, no waiting between them."""
    a = _case([900, 400], ns, 64, 64, seed=105)
    b = _case([300], [5], 16, 64, seed=106)
    want = [_run(*_pick(a, 64)), _run(*_pick(b, 64))]
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    args = [(x[0], x[1], dev(x[2]), 64, dev(x[3]), dev(x[4])) for x in (a, b)]
    for _ in range(4):
        got = [m.smla_chunk_attention(*x, softmax_scale=SCALE, workspace=ws) for x in args]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


@pytest.mark.parametrize("T", [6, 150])
def test_offsets_that_decrease_are_refused_on_the_device(T):
    """Sequences that list the same entries over and over bring more tiles than a workspace holds."""
    H, page, B = 64, 16, 33
    pool = random_pool(8, page, 61)
    table = dev(np.tile(np.arange(8, dtype=np.int32), (B, 1)))
    cu = np.zeros(B + 1, dtype=np.int32)
    cu[1::2] = T
    q = torch.randn((T, H, 512), device="cuda").to(torch.bfloat16)
    out = torch.full((T, H, 448), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 7.0, dtype=torch.float32, device="cuda")
    m.smla_chunk_attention(q, pool, table, page, dev(cu), dev(np.full(B, 128, dtype=np.int32)), out=out, lse=lse)
    assert m.smla_device_status(clear=True) == -7
    assert bool((out == 7).all()) and bool((lse == 7).all())


@pytest.mark.parametrize("cap", [5.0, 30.0, 1000.0])
@pytest.mark.parametrize("B,n", [(64, 1), (2, 32)])
def test_capped_scores_keep_their_digits(B, n, cap):
    """Tokens that see one position, whose score is one exact product: lse is the capped score.
    Relative error: 9e-9 of the series, or past z = 1/4 the exponential form, 1 - 2 / (1 + e): two
    steps of 2^-23 each of the exponential and of the quotient, which are 0.47 e and 0.75 there, over
    tanh(1/4) = 0.245: 5 * 2^-22; a dozen 32-bit roundings of 2^-24 and the conversions to and from
    log2: below 2^-19 together."""
    H, page = 16, 4
    rows = torch.zeros((B * page, ROW), dtype=torch.uint8, device="cuda")
    rows[:, 448:455] = 127
    rows[:, 0] = 0x38                                       # e4m3 1.0
    lens = np.full(B, n, dtype=np.int32)
    table = np.arange(B, dtype=np.int32)[:, None].repeat(-(-n // page), axis=1)
    cu = (np.arange(B + 1) * n).astype(np.int32)
    x = torch.cat([torch.logspace(-3, 2, B * n * H // 2), -torch.logspace(-3, 2, B * n * H // 2)])
    q = torch.zeros((B * n, H, 512), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = x.view(B * n, H).to(torch.bfloat16).cuda()
    m.smla_device_status(clear=True)
    out, lse = m.smla_chunk_attention(q, rows, dev(table), page, dev(cu), dev(lens), softmax_scale=1.0, logit_cap=cap,
                                      vis_begin=dev(np.zeros(B * n, np.int32)), vis_end=dev(np.ones(B * n, np.int32)))
    assert m.smla_device_status(clear=True) == 0
    want = cap * torch.tanh(q[:, :, 0].double() / cap)
    assert ((lse.double() - want).abs() <= 2.0 ** -19 * want.abs()).all()
    assert torch.equal(out[:, :, 0].float(), torch.ones_like(lse)) and not out[:, :, 1:].any()


@pytest.mark.parametrize("ns,H", [([1, 1], 64), ([40, 30], 16)])
@pytest.mark.parametrize("block", [0, 1])
def test_a_wait_that_runs_out_reports_and_the_next_call_is_right(ns, H, block):
    """One warp keeps a signal back (nothing faults): the waits for it end after about a second, the
    call returns, and the next one on the same context is right."""
    page = 16
    q, pool, table, cu, lens = _case([3000, 20000], ns, H, page, 77)
    lib = m._lib.load()
    m.smla_device_status(clear=True)
    assert lib.smla_test_inject_fault(block) == 0
    try:
        m.smla_chunk_attention(q, pool, dev(table), page, dev(cu), dev(lens))
        torch.cuda.synchronize()
        assert m.smla_device_status(clear=True) == m._lib.SMLA_ERR_TIMEOUT
    finally:
        assert lib.smla_test_inject_fault(-1) == 0
    _check(q, pool, table, page, cu, lens)
