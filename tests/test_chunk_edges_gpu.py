"""Chunk attention at the edges of what its arguments allow: masks, lengths and offsets at the
ends of their type, caps far below the scale, values next to bf16's largest, tables that can
hold more than a call is told of.  Tolerances are derived in _cache_helpers, or beside the test."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_03_gb300 as m

from _cache_helpers import ROW, SCALE, check_chunk, chunk_reference, dev, pack_rows, random_pool, tables

pytestmark = pytest.mark.gpu

LOW, HIGH = -2 ** 31, 2 ** 31 - 1


def _case(lens, n, H, page, seed):
    """A batch whose sequences bring n tokens each: 1 to 3 of 64 heads go to single SMs, 140 to
    pairs."""
    num_pages = sum(-(-L // page) for L in lens) + 2
    pool, table = random_pool(num_pages, page, seed), tables(lens, page, num_pages, seed)
    cu = (np.arange(len(lens) + 1) * n).astype(np.int32)
    q = torch.randn(int(cu[-1]), H, 512, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
    return q, pool, table, cu, np.array(lens, np.int32)


def _call(q, pool, table, page, cu, lens, status=0, **kw):
    m.smla_device_status(clear=True)
    kw = {k: dev(v) if isinstance(v, np.ndarray) else v for k, v in kw.items()}
    kw.setdefault("softmax_scale", SCALE)
    got = m.smla_chunk_attention(q, pool, dev(table), page, dev(cu), dev(lens), **kw)
    assert m.smla_device_status(clear=True) == status
    return got


@pytest.mark.parametrize("n", [1, 140])
@pytest.mark.parametrize("first", [True, False])
def test_lengths_as_large_as_their_type(n, first):
    """A length of 2^31 - 1 counts 2^25 blocks: cut to what the bound on the tokens leaves (9 blocks
    here, 7 behind the other sequence's 2) and reported; the sequence behind it finds no room."""
    page, H = 64, 64
    q, pool, table, cu, _ = _case([576, 100] if first else [100, 576], n, H, page, 3)
    lens = np.array([HIGH, 100] if first else [100, HIGH], np.int32)
    got = _call(q, pool, table, page, cu, lens, status=-7, max_kv_tokens=448)
    seen = np.array([576, 100] if first else [100, 448], np.int32)
    end = np.full(2 * n, HIGH, np.int32)
    if first:
        table[1] = -1
    else:
        end[:n] = 100 - n + 1 + np.arange(n)
    check_chunk(got, chunk_reference(q, pool, table, page, cu, seen, begin=np.zeros(2 * n, np.int32), end=end))


@pytest.mark.parametrize("n", [1, 140])
def test_lengths_below_zero_count_as_none(n):
    page, H = 64, 64
    q, pool, table, cu, lens = _case([300, 200], n, H, page, 4)
    for low in (-1, LOW):
        lens[0] = low
        got = _call(q, pool, table, page, cu, lens)
        assert not got[0][:n].any() and torch.isneginf(got[1][:n]).all()
        check_chunk(got, chunk_reference(q, pool, table, page, cu, np.maximum(lens, 0)))


@pytest.mark.parametrize("n,H", [(3, 64), (140, 64), (15, 16), (130, 128)])
def test_masks_at_the_ends_of_their_type(n, H):
    """Tokens that see nothing, or everything, by the least and largest numbers there are, in one
    tile with tokens that see an ordinary part of blocks past the first."""
    L, page = 520, 64
    q, pool, table, cu, lens = _case([L], n, H, page, 7 + H)
    pick = [(0, LOW), (200, 500), (HIGH, HIGH), (LOW, HIGH), (HIGH, LOW), (LOW, LOW), (130, 131)]
    begin = np.array([pick[j % 7][0] for j in range(n)], np.int32)
    end = np.array([pick[j % 7][1] for j in range(n)], np.int32)
    got = _call(q, pool, table, page, cu, lens, vis_begin=begin, vis_end=end)
    check_chunk(got, chunk_reference(q, pool, table, page, cu, lens, begin=begin, end=end))


@pytest.mark.parametrize("T", [2, 140])
@pytest.mark.parametrize("offsets", [lambda T: [0, T + 10], lambda T: [-3, T], [0, 1, HIGH], [LOW, 0, 1],
                                     lambda T: [0, T, 0, T], lambda T: [0, T + 1, T], lambda T: [1, 0, T],
                                     lambda T: [T + 1, T + 1]])
def test_offsets_out_of_order_or_not_of_q_write_nothing(T, offsets):
    """Also those few enough to fit the workspace's room for tiles."""
    H, page, L = 64, 16, 300
    cu = np.array(offsets(T) if callable(offsets) else offsets, np.int32)
    B = len(cu) - 1
    q, pool, table, _, lens = _case([L] * B, T, H, page, 61)
    q = q[:T].contiguous()
    out = torch.full((T, H, 448), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 7.0, dtype=torch.float32, device="cuda")
    _call(q, pool, table, page, cu, lens, status=-7, out=out, lse=lse)
    assert bool((out == 7).all()) and bool((lse == 7).all())


@pytest.mark.parametrize("T", [3, 140])
def test_offsets_at_the_ends_of_q_are_in_order(T):
    """Empty sequences before the first entry and behind the last one."""
    H, page = 64, 16
    q, pool, table, _, lens = _case([300, 200, 100, 50], T, H, page, 62)
    q = q[:T].contiguous()
    cu = np.array([0, 0, T, T, T], np.int32)
    got = _call(q, pool, table, page, cu, lens)
    check_chunk(got, chunk_reference(q, pool, table, page, cu, lens))


@pytest.mark.parametrize("scale,cap", [(1.0, 1e-30), (1.0, 1e-7), (1.0, 1e30), (2.0 ** 33, 5.0), (2.0 ** 33, 30.0),
                                       (2.0 ** 33, 1e-7), (2.0 ** -33, 5.0), (2.0 ** 60, 1e-3), (2.0 ** -40, 1e4)])
@pytest.mark.parametrize("B,n", [(64, 1), (2, 32)])
def test_caps_far_from_the_scale(B, n, scale, cap):
    """Tokens that see one position, whose score is one exact product (the scales are powers of two):
    lse is the capped score, also where the score is 0 and where scale / cap has no eighth power in
    32 bits.  Relative error: past z = 1/4 the exponential form, 1 - 2 / (1 + e): two steps of 2^-23
    each of the exponential and of the quotient, which are 0.47 e and 0.75 there, over tanh(1/4) =
    0.245: 5 * 2^-22; the series 9e-9; a dozen 32-bit roundings of 2^-24 and the conversions to and
    from log2: below 2^-19 together."""
    H, page = 16, 4
    rows = torch.zeros((B * page, ROW), dtype=torch.uint8, device="cuda")
    rows[:, 448:455] = 127
    rows[:, 0] = 0x38                                       # e4m3 1.0
    lens = np.full(B, n, np.int32)
    table = np.arange(B, dtype=np.int32)[:, None].repeat(-(-n // page), axis=1)
    cu = (np.arange(B + 1) * n).astype(np.int32)
    half = torch.logspace(-3, 2, B * n * H // 2, dtype=torch.float64) * (cap / scale)
    x = torch.cat([half, -half])
    x[::5] = 0
    x = x[torch.randperm(x.numel(), generator=torch.Generator().manual_seed(1))]
    q = torch.zeros((B * n, H, 512), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = x.view(B * n, H).to(torch.bfloat16).cuda()
    out, lse = _call(q, rows, table, page, cu, lens, softmax_scale=scale, logit_cap=cap,
                     vis_begin=np.zeros(B * n, np.int32), vis_end=np.ones(B * n, np.int32))
    want = cap * torch.tanh(q[:, :, 0].double() * scale / cap)
    assert ((lse.double() - want).abs() <= 2.0 ** -19 * want.abs()).all()
    assert torch.equal(out[:, :, 0].float(), torch.ones_like(lse)) and not out[:, :, 1:].any()


@pytest.mark.parametrize("H", [16, 64])
def test_tables_that_hold_more_than_the_largest_bound(H):
    """The default bound is what the table can hold, kept within what the call takes."""
    page, L = 4096, [5000, 300]
    q, pool, table, cu, lens = _case(L, 1, H, page, 71)
    wide = np.full((2, (1 << 17) + 1), -1, np.int32)          # 2 * 131,073 pages of 4,096: 2^30 and 8,192
    wide[:, :table.shape[1]] = table
    assert wide.size * page > 1 << 30
    got = _call(q, pool, wide, page, cu, lens)
    check_chunk(got, chunk_reference(q, pool, table, page, cu, lens))


@pytest.mark.parametrize("n,H", [(2, 64), (40, 64), (15, 16)])
def test_values_next_to_the_largest_of_bf16(n, H):
    """1.8 * 2^127 in a group is stored with the scale byte 247, and values up to 240 * 2^120 are
    numbers: rows of any scale byte count as finite while all their values are.  One block, so that
    no weight passes 1, and one such row a group, so that the sums stay below 2^128."""
    L, page = 50, 64
    q, pool, table, cu, lens = _case([L], n, H, page, 23)
    q[:, :, 64:320] = 0
    x = torch.randn(L, 512, generator=torch.Generator().manual_seed(4))
    x[:, 64:320] = 0
    x[7, 70], x[9, 130] = 1.8 * 2.0 ** 127, -1.85 * 2.0 ** 127
    rows = pack_rows(x.to(torch.bfloat16))
    assert rows[7, 449] == 247 and rows[9, 450] == 247
    rows[11, 451], rows[11, 192:256] = 254, 0x3F                # 1.875 * 2^127
    rows[11, 200:230] = 0
    rows[12, 452] = 254                                         # zeros with the largest scale
    at = torch.as_tensor(table[0].astype(np.int64)[np.arange(L) // page] * page + np.arange(L) % page, device="cuda")
    pool[at] = dev(rows)
    got = _call(q, pool, table, page, cu, lens)
    check_chunk(got, chunk_reference(q, pool, table, page, cu, lens))
    # one step more, and the row is not finite: who sees it gets NaN
    begin, end = np.arange(n, dtype=np.int32), np.full(n, L, np.int32)
    for row, col, group, byte, code in ((7, 70, 449, 247, 0x78), (12, 256, 452, 254, 0x40), (12, 257, 452, 248, 0x70)):
        bad = rows.copy()
        bad[row, col], bad[row, group] = code, byte
        pool[at] = dev(bad)
        out, lse = _call(q, pool, table, page, cu, lens, vis_begin=begin, vis_end=end)
        sees = torch.arange(n, device="cuda") <= row
        assert torch.isnan(out[sees].float()).all() and torch.isnan(lse[sees]).all()
        clean = pool.clone()
        clean[at[row]] = 0
        ref = chunk_reference(q, clean, table, page, cu, lens, begin=begin, end=end)
        ref[0][sees] = ref[1][sees] = float("nan")              # (not compared)
        check_chunk((out, lse), ref)


@pytest.mark.parametrize("cap", [1e-7, 3e38])
@pytest.mark.parametrize("n", [1, 140])
def test_the_least_and_the_largest_caps(n, cap):
    """All positions weigh the same, or the cap does nothing; a query of zeros among the others."""
    q, pool, table, cu, lens = _case([400], n, 64, 64, 17)
    q[0, 5] = 0
    got = _call(q, pool, table, 64, cu, lens, logit_cap=cap)
    ref = chunk_reference(q, pool, table, 64, cu, lens, SCALE, 1e-7 if cap < 1 else 0.0)
    check_chunk(got, ref)
