"""Rows of 4-bit values: what the append writes, the read returns and the page calls move, byte by
byte, and attention over them (chunks, single tokens, lists of rows and positions) against the
definition in 64 bits.  Tolerances: _cache_helpers."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_03_gb300 as m

from _cache_helpers import (PageModel, ROW, SCALE, check_chunk, check_pages, chunk_reference, dev, pack_rows, random_pool, tables)
from _rows4_helpers import ROW4, chunk_reference4, dequantize4, pack_rows4, random_pool4

pytestmark = pytest.mark.gpu


def _ints(v):
    return dev(np.asarray(v, np.int32))


def _append_case(lens, ns, page, seed, stride=ROW4, lead=0, pad=0):
    rng = np.random.default_rng(seed)
    num_pages = sum(-(-L // page) for L in lens) + 3
    pool = random_pool4(num_pages, page, seed, stride, lead)
    table = tables(lens, page, num_pages, seed)
    wide = torch.as_tensor(rng.standard_normal((sum(ns), 512 + pad)) * np.exp2(rng.integers(-9, 9, (sum(ns), 1))),
                           dtype=torch.float32).to(torch.bfloat16).cuda()
    return pool, table, wide[:, :512], np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)


def _rows(table, lens, cu, page):
    return np.concatenate([[table[b, p // page] * page + p % page for p in range(L - (cu[b + 1] - cu[b]), L)]
                           for b, L in enumerate(lens)]).astype(np.int64)


@pytest.mark.parametrize("lens,ns,page,stride,lead,pad", [
    ([1], [1], 1, ROW4, 0, 0),
    ([5, 40, 17], [5, 1, 17], 16, ROW4, 16, 0),
    ([100, 33, 64, 7], [64, 0, 1, 7], 48, 384, 16, 8),
    ([130] * 40, [3] * 40, 64, 512, 0, 0),
    ([70 + i for i in range(70)], [i % 3 for i in range(70)], 7, ROW4, 48, 16),
])
def test_append_and_read(lens, ns, page, stride, lead, pad):
    pool, table, kv, cu = _append_case(lens, ns, page, 10 + page, stride, lead, pad)
    want = pool.cpu().numpy().copy()
    at = _rows(table, lens, cu, page)
    want[at, :ROW4] = pack_rows4(kv)
    m.smla_device_status(clear=True)
    args = (dev(table), page, _ints(cu), _ints(lens))
    m.smla_cache_append(kv, pool, *args)
    assert m.smla_device_status(clear=True) == 0
    assert np.array_equal(pool.cpu().numpy(), want)
    got = m.smla_cache_read(pool, *args, kv.shape[0])
    assert m.smla_device_status(clear=True) == 0
    nope, rope = dequantize4(want[at])
    assert np.array_equal(got.double().cpu().numpy(), np.concatenate([nope, rope], axis=1))


def test_append_extreme_values():
    """Zeros (and -0), the scale borders 6 * 2^e and just above, ties, bf16's largest and smallest,
    subnormals; a group with an infinity or a NaN is NaN and reported."""
    page, n = 16, 14
    x = torch.zeros(n, 512)
    x[0, 3] = -0.0
    x[1, :32] = torch.linspace(-6, 6, 32)
    x[2, 0], x[2, 32], x[2, 64] = 6.0, 6.03125, 5.96875
    x[3, :448] = 2.2e38
    x[4, :448] = 1.1754943508222875e-38
    x[5, :448] = 9.183549615799121e-41
    x[6, 0] = 6.0
    x[6, 1:15] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0])
    x[6, 15:22] = torch.tensor([0.251953125, 0.74609375, 1.2578125, 1.7421875, 2.515625, 3.484375, 5.03125])
    x[7, 100], x[7, 101] = float("inf"), 3.0
    x[8, 200], x[8, 201] = float("nan"), -5.0
    x[9, 300], x[9, 301] = float("-inf"), 1e-3
    x[10, 448:] = float("nan")
    x[11, 447], x[11, 0] = -1.0, 2.0 ** -20
    x[12, 0], x[12, 1] = 3.3895313892515355e38, 1e38
    x[13, 31], x[13, 32] = 100.0, 0.01
    kv = x.to(torch.bfloat16).cuda()
    pool = torch.full((2 * page, ROW4), 7, dtype=torch.uint8, device="cuda")
    args = (_ints([[1]]), page, _ints([0, n]), _ints([n]))
    m.smla_device_status(clear=True)
    m.smla_cache_append(kv, pool, *args)
    assert m.smla_device_status(clear=True) == -8
    got, want = pool.cpu().numpy(), pack_rows4(kv)
    assert (got[:page] == 7).all() and (got[page + n:] == 7).all()
    assert np.array_equal(got[page:page + n], want)
    back = m.smla_cache_read(pool, *args, n).double().cpu().numpy()
    nope, rope = dequantize4(want)
    expect = np.concatenate([nope, rope], axis=1)
    expect[np.abs(expect) >= 2.0 ** 128] = np.inf          # stored as 2^128, past bf16
    assert np.array_equal(back, expect, equal_nan=True)


@pytest.mark.parametrize("value,code", [(1.7421875 * 2.0 ** 127, 0), (1.75 * 2.0 ** 127, -8)])
def test_append_at_the_border_of_2_to_128(value, code):
    kv = torch.zeros(1, 512)
    kv[0, 5] = value
    pool = torch.zeros(4, ROW4, dtype=torch.uint8, device="cuda")
    m.smla_device_status(clear=True)
    m.smla_cache_append(kv.to(torch.bfloat16).cuda(), pool, _ints([[0]]), 4, _ints([0, 1]), _ints([1]))
    assert m.smla_device_status(clear=True) == code


def test_read_of_8_bit_rows():
    page, lens, ns = 16, [40, 5, 100], [40, 0, 61]
    pool = random_pool(12, page, 3)
    table = tables(lens, page, 12, 3)
    cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    out = torch.full((120, 520), 9.0, dtype=torch.bfloat16, device="cuda")
    m.smla_device_status(clear=True)
    got = m.smla_cache_read(pool, dev(table), page, _ints(cu), _ints(lens), 120, out=out[:, :512])
    assert m.smla_device_status(clear=True) == 0
    import oracle.mla_oracle as O
    nope, rope = O.dequantize_rows(pool.cpu().numpy()[_rows(table, lens, cu, page)])
    assert np.array_equal(got[:101].double().cpu().numpy(), np.concatenate([nope, rope], axis=1))
    assert (out[101:] == 9).all() and (out[:, 512:] == 9).all()


def test_read_and_append_skip_tokens_without_a_place():
    page = 8
    pool = random_pool4(6, page, 3)
    before = pool.cpu().numpy().copy()
    kv = torch.randn(20, 512, device="cuda").to(torch.bfloat16)
    args = (_ints([[0, -1, 2], [9, 3, -1], [4, 5, 1]]), page, _ints([2, 6, 10, 12]), _ints([16, 7, 25]))
    m.smla_device_status(clear=True)
    out = torch.full((20, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    m.smla_cache_read(pool, *args, 20, out=out)
    assert m.smla_device_status(clear=True) == -7
    nope, rope = dequantize4(before[15:16])
    assert np.array_equal(out[10].double().cpu().numpy(), np.concatenate([nope, rope], axis=1)[0])
    rest = [t for t in range(20) if t != 10]
    assert (out[rest] == 3).all()
    m.smla_cache_append(kv, pool, *args)
    assert m.smla_device_status(clear=True) == -7
    before[15] = pack_rows4(kv[10:11])[0]
    assert np.array_equal(pool.cpu().numpy(), before)


@pytest.mark.parametrize("stride,lead", [(ROW4, 0), (400, 16)])
def test_page_calls_move_whole_rows_and_nothing_else(stride, lead):
    page, num_pages, rows, width = 24, 90, 6, 9
    pool = random_pool4(num_pages, page, 5, stride, lead)
    lens = [page * 3 + 7, 50, page * 8, 0, 0, 1]
    table = tables(lens, page, num_pages, 6, extra=width - 8)
    ref = np.zeros(num_pages, np.int32)
    ref[table[table >= 0]] = 1
    model = PageModel(ref, table, lens, page)
    want = pool.cpu().numpy().copy()
    r, t, l = dev(ref), dev(table), _ints(lens)
    m.smla_device_status(clear=True)
    m.smla_cache_fork(pool, page, r, t, l, _ints([0, 1, 0]), _ints([3, 4, 5]))
    model.free([5])                                   # the model's child rows are free rows
    model.ref[table[5, 0]] += 1                       # ... the call's is overwritten, not freed
    model.fork([0, 1, 0], [3, 4, 5])
    check_pages(model, r, t, l)
    info = m.smla_cache_compact(pool, page, r, t)
    assert info.cpu().tolist() == list(model.compact())
    check_pages(model, r, t, l)
    for a, b, k in model.copies:
        want[b * page:b * page + k, :ROW4] = want[a * page:a * page + k, :ROW4]
    assert m.smla_device_status(clear=True) == 0
    assert np.array_equal(pool.cpu().numpy()[:, :ROW4], want[:, :ROW4])
    assert (pool.cpu().numpy()[:, ROW4:] == 0xA5).all()


# ---------------------------------------------------------------- attention
def _case(lens, ns, H, page, seed, stride=ROW4, lead=0, mult=1.0, extra=1):
    num_pages = sum(-(-max(L, 0) // page) for L in lens) + 2
    pool = random_pool4(num_pages, page, seed, stride, lead, mult)
    table = tables(lens, page, num_pages, seed, extra)
    cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((max(1, int(cu[-1])), H, 512), generator=g).to(torch.bfloat16).cuda()
    return q, pool, table, page, cu, np.array(lens, np.int32)


def _run(q, pool, table, page, cu, lens, cap=0.0, slopes=None, begin=None, end=None, status=0, **kw):
    m.smla_device_status(clear=True)
    got = m.smla_chunk_attention(q, pool, dev(table), page, dev(cu), dev(lens), softmax_scale=SCALE, logit_cap=cap,
                                 slopes=slopes, vis_begin=None if begin is None else dev(begin),
                                 vis_end=None if end is None else dev(end), **kw)
    assert m.smla_device_status(clear=True) == status
    return got


def _check(q, pool, table, page, cu, lens, cap=0.0, slopes=None, begin=None, end=None, **kw):
    got = _run(q, pool, table, page, cu, lens, cap, slopes, begin, end, **kw)
    check_chunk(got, chunk_reference4(q, pool, table, page, cu, lens, SCALE, cap, slopes, begin, end))
    return got


@pytest.mark.parametrize("lens,ns,H,page", [
    ([1], [1], 64, 1),
    ([1, 2, 3], [1, 1, 3], 16, 1),
    ([64, 63, 65, 0, 1], [1, 1, 1, 0, 1], 64, 16),
    ([1001, 700, 30], [4, 1, 4], 64, 16),
    ([300, 5000], [1, 1], 32, 48),
    ([257], [3], 128, 64),
    ([700, 450], [200, 37], 16, 100),
    ([513, 80], [130, 80], 32, 64),
    ([400], [140], 128, 7),
    ([2500, 0, 1300, 90], [64, 0, 33, 90], 64, 64),
])
def test_causal(lens, ns, H, page):
    _check(*_case(lens, ns, H, page, seed=H + page + len(lens)))


@pytest.mark.parametrize("lens,ns,H,page", [([900, 333], [40, 70], 64, 48), ([600, 77, 1], [1, 1, 1], 64, 16),
                                            ([500], [300], 16, 64)])
def test_masks_cap_and_bias(lens, ns, H, page):
    c = _case(lens, ns, H, page, seed=3 * H)
    rng = np.random.default_rng(H)
    T = sum(ns)
    begin, end = (rng.integers(-20, max(lens) + 40, T).astype(np.int32) for _ in range(2))
    _check(*c, begin=begin, end=end)
    slopes = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H).float()
    _check(*c, cap=5.0, slopes=slopes)


@pytest.mark.parametrize("stride,lead", [(384, 16), (512, 0), (496, 48)])
@pytest.mark.parametrize("n", [1, 135])
def test_strided_pools(stride, lead, n):
    _check(*_case([333], [n], 64, 48, seed=41, stride=stride, lead=lead))


@pytest.mark.parametrize("n", [1, 135])
def test_scale_bytes_of_every_size(n):
    """Bytes past 128 need a second factor, those next to 0 make subnormals."""
    q, pool, table, page, cu, lens = _case([400], [n], 64, 64, seed=43)
    rows = pool.cpu().numpy()
    rng = np.random.default_rng(3)
    rows[::3, 224:238] = rng.integers(120, 140, size=rows[::3, 224:238].shape)
    rows[1::5, 224:238] = rng.integers(0, 30, size=rows[1::5, 224:238].shape)
    pool.copy_(torch.as_tensor(rows))
    _check((q.float() * 2.0 ** -12).to(torch.bfloat16), pool, table, page, cu, lens)


@pytest.mark.parametrize("n", [1, 135])
def test_values_next_to_bf16_largest(n):
    """Scale bytes 252 .. 254 with nibbles that stay within bf16 count as finite; ones past it do not."""
    L, page = 130, 64
    q, pool, table, page, cu, lens = _case([L], [n], 64, page, seed=44)
    rows = pool.cpu().numpy()
    row = table[0, 0] * page + 5
    tiny = (q.float() * 2.0 ** -126).to(torch.bfloat16)
    begin = np.full(n, 0, np.int32)
    for byte, nibble, finite in [(252, 7, True), (253, 5, True), (253, 6, False), (254, 3, True), (254, 4, False),
                                 (255, 0, False)]:
        r = rows.copy()
        r[:, :224] = 0
        r[:, 240:] = 0
        r[row, :224] = nibble * 17
        r[row, 224:238] = byte
        pool.copy_(torch.as_tensor(r))
        out, lse = _run(tiny, pool, table, page, cu, lens, begin=begin, end=np.full(n, 6, np.int32))
        assert torch.isfinite(lse).all() == finite, (byte, nibble)
        if not finite:
            assert torch.isnan(lse).all() and torch.isnan(out.float()).all()


@pytest.mark.parametrize("what", ["rope_nan", "rope_inf", "scale_255"])
@pytest.mark.parametrize("n", [1, 135])
def test_rows_that_are_not_finite(what, n):
    L, page = 500, 48
    q, pool, table, page, cu, lens = _case([L], [n], 64, page, seed=45)
    clean = pool.clone()
    rows = pool.cpu().numpy()
    at = table[0, 300 // page] * page + 300 % page
    if what == "scale_255":
        rows[at, 224 + 9] = 255
    else:
        rows[at, 240 + 2 * 17:240 + 2 * 17 + 2] = np.array([0x7FC1 if what == "rope_nan" else 0xFF80], "<u2").view(np.uint8)
    pool.copy_(torch.as_tensor(rows))
    end = np.where(np.arange(n) % 2 == 0, 300, 301).astype(np.int32)
    out, lse = _run(q, pool, table, page, cu, lens, end=end)
    sees = torch.as_tensor(end > 300, device="cuda")
    assert torch.isnan(lse[sees]).all() and torch.isnan(out[sees].float()).all()
    ref = chunk_reference4(q, clean, table, page, cu, lens, SCALE, end=end)
    check_chunk((out[~sees], lse[~sees]), [t[~sees] for t in ref])


@pytest.mark.parametrize("n", [1, 140])
def test_unmapped_pages_and_bad_ids(n):
    q, pool, table, page, cu, lens = _case([700], [n], 64, 64, seed=46)
    table[0, 3] = -1
    _check(q, pool, table, page, cu, lens)
    table[0, 5] = pool.shape[0] // page
    _check(q, pool, table, page, cu, lens, status=-7)


# ---------------------------------------------------------------- lists of rows
def _sparse_reference(q, pool, table, indices):
    """Each query as a sequence of pages of one row."""
    B, k = indices.shape
    rows = indices.astype(np.int64) if table is None else None
    if table is not None:
        t, page = table
        rows = np.full(indices.shape, -1, np.int64)
        for b in range(B):
            for i, p in enumerate(indices[b]):
                if p >= 0 and p // page < t.shape[1] and t[b, p // page] >= 0:
                    rows[b, i] = t[b, p // page] * page + p % page
    cu = np.arange(B + 1).astype(np.int32)
    return chunk_reference4(q, pool, rows.astype(np.int32), 1, cu, np.full(B, k, np.int32))


def _sparse_case(B, H, k, seed, num_rows=3000, masked=0.1, stride=ROW4):
    rng = np.random.default_rng(seed)
    pool = random_pool4(num_rows, 1, seed, stride)
    idx = rng.integers(0, num_rows, (B, k)).astype(np.int32)
    idx[rng.random((B, k)) < masked] = -1
    q = torch.randn((B, H, 512), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
    return q, pool, idx


@pytest.mark.parametrize("H", [16, 32, 64, 128])
@pytest.mark.parametrize("B,k", [(1, 1), (3, 63), (2, 64), (5, 65), (1, 1500), (40, 300)])
def test_sparse_decode(H, B, k):
    q, pool, idx = _sparse_case(B, H, k, H + k)
    m.smla_device_status(clear=True)
    got = m.sparse_mla_decode(q, pool, dev(idx), SCALE)
    assert m.smla_device_status(clear=True) == 0
    check_chunk(got, _sparse_reference(q, pool, None, idx))


def test_sparse_decode_of_nothing_and_of_a_hole():
    q, pool, idx = _sparse_case(3, 64, 200, 7)
    idx[0] = -1
    idx[1, 64:128] = -1
    got = m.sparse_mla_decode(q, pool, dev(idx), SCALE)
    check_chunk(got, _sparse_reference(q, pool, None, idx))
    assert (got[0][0] == 0).all() and torch.isneginf(got[1][0]).all()


def test_sparse_decode_masks_and_reports_rows_past_the_cache():
    q, pool, idx = _sparse_case(2, 64, 150, 8, num_rows=500, stride=384)
    bad = idx.copy()
    bad[0, 17], bad[1, 149] = 500, 2 ** 31 - 1
    idx[0, 17] = idx[1, 149] = -1
    m.smla_device_status(clear=True)
    got = m.sparse_mla_decode(q, pool, dev(bad), SCALE)
    assert m.smla_device_status(clear=True) == -7
    check_chunk(got, _sparse_reference(q, pool, None, idx))


@pytest.mark.parametrize("page", [1, 16, 100])
def test_sparse_decode_of_pages(page):
    lens, H, k = [900, 30, 444], 64, 130
    num_pages = sum(-(-L // page) for L in lens) + 2
    pool = random_pool4(num_pages, page, page)
    table = tables(lens, page, num_pages, page)
    rng = np.random.default_rng(page)
    idx = np.stack([rng.integers(-3, L, k) for L in lens]).astype(np.int32)
    idx = np.maximum(idx, -1)
    q = torch.randn((3, H, 512), generator=torch.Generator().manual_seed(page)).to(torch.bfloat16).cuda()
    m.smla_device_status(clear=True)
    got = m.sparse_mla_decode_paged(q, pool, dev(table), page, dev(idx), SCALE)
    assert m.smla_device_status(clear=True) == 0
    check_chunk(got, _sparse_reference(q, pool, (table, page), idx))
    # unmapped: masked; past the table or the pool: masked and reported
    bad = table.copy()
    bad[0, 0] = -1
    got = m.sparse_mla_decode_paged(q, pool, dev(bad), page, dev(idx), SCALE)
    assert m.smla_device_status(clear=True) == 0
    check_chunk(got, _sparse_reference(q, pool, (bad, page), idx))
    over = idx.copy()
    over[1, 3] = table.shape[1] * page
    over[2, 5] = 2 ** 31 - 1
    idx[1, 3] = idx[2, 5] = -1
    got = m.sparse_mla_decode_paged(q, pool, dev(table), page, dev(over), SCALE)
    assert m.smla_device_status(clear=True) == -7
    check_chunk(got, _sparse_reference(q, pool, (table, page), idx))
    bad = table.copy()
    bad[0, 0] = num_pages
    m.sparse_mla_decode_paged(q, pool, dev(bad), page, dev(np.zeros_like(idx)), SCALE)
    assert m.smla_device_status(clear=True) == -7


def test_sparse_decode_replays_and_repeats():
    q, pool, idx = _sparse_case(9, 64, 700, 11)
    i = dev(idx)
    p = m.make_params(9, 64, 700, pool.shape[0], ROW4, SCALE)
    ws = torch.empty(m.smla_workspace_size(p), dtype=torch.uint8, device="cuda")
    out, lse = m.sparse_mla_decode(q, pool, i, SCALE, workspace=ws)
    again = m.sparse_mla_decode(q, pool, i, SCALE)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        m.sparse_mla_decode(q, pool, i, SCALE, out=out, lse=lse, workspace=ws)
    for seed in (12, 13):
        _, _, idx = _sparse_case(9, 64, 700, seed)
        i.copy_(dev(idx))
        g.replay()
        torch.cuda.synchronize()
        check_chunk((out, lse), _sparse_reference(q, pool, None, idx))


def test_rows_past_32_bits_of_offset():
    """Rows whose byte offset passes 2^32: 12 million rows of 368 bytes."""
    n = 12_000_000
    if torch.cuda.mem_get_info()[0] < n * ROW4 + (2 << 30):
        pytest.skip("not enough memory")
    pool = torch.zeros((n, ROW4), dtype=torch.uint8, device="cuda")
    last = random_pool4(64, 1, 9)
    pool[n - 64:] = last
    q = torch.randn((1, 64, 512), generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    idx = np.arange(n - 64, n)[None].astype(np.int32)
    got = m.sparse_mla_decode(q, pool, dev(idx), SCALE)
    want = m.sparse_mla_decode(q, last, dev(np.arange(64)[None].astype(np.int32)), SCALE)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("H,lens,ns", [
    (64, [700 + 331 * i for i in range(32)], [1] * 32),
    (16, [1 + 97 * i for i in range(32)], [1] * 32),
    (128, [9000, 3, 64, 65, 0, 2000], [2, 3, 1, 2, 0, 3]),
    (32, [40000], [5]),
    (64, [0] * 32, [1] * 32),
])
@pytest.mark.parametrize("bits", [8, 4])
def test_an_empty_sequence_more_changes_no_bit(bits, H, lens, ns):
    """The plan that each SM works out for up to 32 sequences and tiles is the one that a kernel makes for more."""
    page = 64
    num_pages = sum(-(-L // page) for L in lens) + 2
    pool = (random_pool if bits == 8 else random_pool4)(num_pages, page, 5)
    table = tables(lens, page, num_pages, 5)
    T = sum(ns)
    cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    q = torch.randn(T, H, 512, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).cuda()
    begin = torch.arange(T, dtype=torch.int32, device="cuda") * 13
    end = torch.full((T,), 30000, dtype=torch.int32, device="cuda")
    more = 33 - len(lens)
    for kw in ({}, {"vis_begin": begin, "vis_end": end}):
        few = m.smla_chunk_attention(q, pool, dev(table), page, dev(cu), dev(np.array(lens, np.int32)), softmax_scale=SCALE,
                                     max_kv_tokens=sum(lens) + 1, **kw)
        many = m.smla_chunk_attention(q, pool, dev(np.concatenate([table, np.full((more, table.shape[1]), -1, np.int32)])), page,
                                      dev(np.concatenate([cu, np.full(more, T, np.int32)])),
                                      dev(np.array(lens + [0] * more, np.int32)), softmax_scale=SCALE,
                                     max_kv_tokens=sum(lens) + 1, **kw)
        # One warp of the merge adds up a row's parts, or eight where 4 * (T H / 64 + sequences) is within the 152 SMs: six
        # sequences of 11 tokens of 128 heads are, 33 of them are not.  The order of a sum then differs, the plan does not.
        tiles = (T * H + 63) // 64
        if (4 * (tiles + len(lens)) <= 152) == (4 * (tiles + 33) <= 152):
            assert torch.equal(few[0].view(torch.int16), many[0].view(torch.int16))
            assert torch.equal(few[1], many[1])
        else:
            masks = {"begin": kw["vis_begin"].cpu().numpy(), "end": kw["vis_end"].cpu().numpy()} if kw else {}
            want = (chunk_reference4 if bits == 4 else chunk_reference)(q, pool, table, page, cu, np.array(lens), **masks)
            check_chunk(few, want)
            check_chunk(many, want)


@pytest.mark.parametrize("cu", [[0, 3, 2, 5], [0, 2, 4, 9], [-1, 2, 4, 5]])
def test_offsets_that_are_wrong_write_nothing(cu):
    pool, table = random_pool4(9, 64, 2), tables([100, 100, 100], 64, 9, 2)
    q = torch.randn(5, 64, 512).to(torch.bfloat16).cuda()
    out, lse = torch.full((5, 64, 448), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((5, 64), 7.0, device="cuda")
    m.smla_device_status(clear=True)
    m.smla_chunk_attention(q, pool, dev(table), 64, dev(np.array(cu, np.int32)), dev(np.array([100] * 3, np.int32)), out=out, lse=lse)
    assert m.smla_device_status(clear=True) == m._lib.SMLA_ERR_INDEX_RANGE
    assert (out == 7).all() and (lse == 7).all()
