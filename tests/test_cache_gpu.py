"""The paged cache's calls on a GPU: append against the definition value by value, the page
calls against a step-by-step model in Python."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_03_gb300 as m

from _cache_helpers import ROW, PageModel, check_pages, dev, pack_rows, random_pool, tables

pytestmark = pytest.mark.gpu


def _append_case(lens, ns, page, seed, stride=ROW, lead=0, kv_pad=0, mult=1.0):
    rng = np.random.default_rng(seed)
    num_pages = sum(-(-L // page) for L in lens) + 3
    pool = random_pool(num_pages, page, seed, stride, lead)
    table = tables(lens, page, num_pages, seed)
    T = sum(ns)
    wide = torch.as_tensor(rng.standard_normal((T, 512 + kv_pad)) * mult * np.exp2(rng.integers(-9, 9, (T, 1))),
                           dtype=torch.float32).to(torch.bfloat16).cuda()
    cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    return pool, table, wide[:, :512], cu


def _expected(pool, table, kv, cu, lens, page):
    want = pool.cpu().numpy().copy()
    rows = pack_rows(kv)
    for b, L in enumerate(lens):
        n = cu[b + 1] - cu[b]
        for j in range(n):
            p = L - n + j
            want[table[b, p // page] * page + p % page, :ROW] = rows[cu[b] + j]
    return want


@pytest.mark.parametrize("lens,ns,page,stride,lead,pad", [
    ([1], [1], 1, ROW, 0, 0),
    ([5, 40, 17], [5, 1, 17], 16, ROW, 0, 0),
    ([100, 33, 64, 7], [64, 0, 1, 7], 48, 600, 8, 8),
    ([130] * 40, [3] * 40, 64, 592, 16, 0),
    ([70 + i for i in range(70)], [i % 3 for i in range(70)], 7, ROW, 8, 16),
])
def test_append_writes_the_defined_bytes_and_nothing_else(lens, ns, page, stride, lead, pad):
    pool, table, kv, cu = _append_case(lens, ns, page, 10 + page, stride, lead, pad)
    want = _expected(pool, table, kv, cu, lens, page)
    m.smla_device_status(clear=True)
    m.smla_cache_append(kv, pool, dev(table), page, dev(cu), dev(np.array(lens, np.int32)))
    assert m.smla_device_status(clear=True) == 0
    assert np.array_equal(pool.cpu().numpy(), want)


def test_append_extreme_values():
    """Zeros (and -0), the scale borders 448 * 2^e and just above, bf16's largest and smallest,
    subnormals, ties; infinities and NaN are stored as NaN and reported."""
    page, n = 16, 12
    x = torch.zeros(n, 512)
    x[0, 3] = -0.0
    x[1, :64] = torch.linspace(-448, 448, 64)
    x[2, 0], x[2, 64], x[2, 128] = 448.0, 450.0, 447.0
    x[3, :448] = 3.3895313892515355e38
    x[4, :448] = 1.1754943508222875e-38
    x[5, :448] = 9.183549615799121e-41
    x[6, 0] = 448.0
    x[6, 1:17] = torch.tensor([17.0, 19.0, 18.0, 2 ** -9, 3 * 2 ** -10, 2 ** -10, 0.75 * 2 ** -9, 5 * 2 ** -10,
                               -17.0, -19.0, 208.0, 216.0, 1.0625, 1.1875, 2 ** -7, 15 * 2 ** -10])
    x[7, 100], x[7, 101] = float("inf"), 3.0
    x[8, 200], x[8, 201] = float("nan"), -5.0
    x[9, 300], x[9, 301] = float("-inf"), 1e-3
    x[10, 448:] = float("nan")
    x[11, 447], x[11, 0] = -1.0, 2.0 ** -20
    kv = x.to(torch.bfloat16).cuda()
    pool = torch.full((2 * page, ROW), 7, dtype=torch.uint8, device="cuda")
    table = np.array([[1]], np.int32)
    m.smla_device_status(clear=True)
    m.smla_cache_append(kv, pool, dev(table), page, dev(np.array([0, n], np.int32)), dev(np.array([n], np.int32)))
    assert m.smla_device_status(clear=True) == -8
    got, want = pool.cpu().numpy(), pack_rows(kv)
    assert (got[:page] == 7).all() and (got[page + n:] == 7).all()
    nan = (want[:, :448] & 0x7F) == 0x7F
    assert np.array_equal((got[page:page + n, :448] & 0x7F) == 0x7F, nan)
    a, b = got[page:page + n].copy(), want.copy()
    a[:, :448][nan] = b[:, :448][nan] = 0        # a NaN's sign carries nothing
    assert np.array_equal(a, b)


def test_append_skips_tokens_without_a_place_and_reports():
    page = 8
    pool = random_pool(6, page, 3)
    before = pool.clone()
    kv = torch.randn(20, 512, device="cuda").to(torch.bfloat16)
    table = np.array([[0, -1, 2], [9, 3, -1], [4, 5, 1]], np.int32)     # 9: past the pool
    lens = np.array([16, 7, 25], np.int32)                              # 25: past a table of 24
    cu = np.array([2, 6, 10, 12], np.int32)                             # 0, 1 and 12.. belong to none
    m.smla_device_status(clear=True)
    m.smla_cache_append(kv, pool, dev(table), page, dev(cu), dev(lens))
    assert m.smla_device_status(clear=True) == -7
    want = before.cpu().numpy().copy()
    want[1 * page + 7] = pack_rows(kv[10:11])[0]                        # position 23 of sequence 2
    assert np.array_equal(pool.cpu().numpy(), want)


def test_append_more_new_tokens_than_the_length():
    pool = random_pool(2, 4, 5)
    before = pool.cpu().numpy().copy()
    kv = torch.randn(5, 512, device="cuda").to(torch.bfloat16)
    m.smla_device_status(clear=True)
    m.smla_cache_append(kv, pool, dev(np.array([[1, 0]], np.int32)), 4, dev(np.array([0, 5], np.int32)),
                        dev(np.array([2], np.int32)))
    assert m.smla_device_status(clear=True) == -7
    before[4:6] = pack_rows(kv[3:5])
    assert np.array_equal(pool.cpu().numpy(), before)


# ---------------------------------------------------------------- page calls
def _state(num_pages, page, R, width, lens, seed, reserve_extra=0):
    rng = np.random.default_rng(seed)
    table = np.full((R, width), -1, dtype=np.int32)
    order = rng.permutation(num_pages)
    ref = np.zeros(num_pages, dtype=np.int32)
    at = 0
    for r, L in enumerate(lens):
        k = min(width, -(-L // page) + (reserve_extra if L else 0))
        table[r, :k] = order[at:at + k]
        ref[order[at:at + k]] = 1
        at += k
    return ref, table, np.array(lens, dtype=np.int32)


@pytest.mark.parametrize("num_pages,page,R,width,seed", [(9, 4, 3, 5, 0), (500, 16, 20, 30, 1),
                                                         (5000, 1, 40, 200, 2), (70000, 64, 300, 33, 3)])
def test_branches_dropped_forked_grown_and_compacted(num_pages, page, R, width, seed):
    """The calls in the order a program makes them, each against the model, and the pool's
    bytes at the end."""
    rng = np.random.default_rng(seed)
    lens = [int(rng.integers(0, max(2, min(width * page, num_pages * page // (2 * R))))) for _ in range(R)]
    lens[0] = max(1, lens[0])
    lens[R - 1] = (lens[0] // page) * page            # no partial page
    ref, table, kv_lens = _state(num_pages, page, R, width, lens, seed)
    pool = torch.randint(0, 256, (num_pages * page, ROW), device="cuda", dtype=torch.uint8)
    want = pool.cpu().numpy().copy().reshape(num_pages, page, ROW)
    model = PageModel(ref, table, lens, page)
    ref, table, kv_lens = dev(ref), dev(table), dev(kv_lens)
    m.smla_device_status(clear=True)
    children = rng.permutation(np.arange(R // 2, R))[:max(1, R // 3)].astype(np.int32)
    parents = rng.integers(0, max(1, R // 2), len(children)).astype(np.int32)
    for _ in range(2):
        m.smla_cache_free(ref, table, kv_lens, dev(children))
        model.free(children)
        check_pages(model, ref, table, kv_lens)
        m.smla_cache_fork(pool, page, ref, table, kv_lens, dev(parents), dev(children))
        model.fork(parents, children)
        check_pages(model, ref, table, kv_lens)
        target = np.minimum(np.array(model.lens) + rng.integers(0, 2 * page + 1, R), width * page).astype(np.int32)
        m.smla_cache_reserve(page, ref, table, dev(target))
        model.reserve(target)
        check_pages(model, ref, table, kv_lens)
    m.smla_cache_free(ref, table, kv_lens, dev(children[::2].copy()))
    model.free(children[::2])
    ref_out, table_out = torch.full_like(ref, -5), torch.full_like(table, -5)
    moved = PageModel(model.ref, model.table, model.lens, page)
    n, k = moved.compact()
    keep = pool.clone()
    info = m.smla_cache_compact(keep, page, ref, table, ref_count_out=ref_out, block_table_out=table_out)
    assert info.cpu().tolist() == [n, k]
    check_pages(moved, ref_out, table_out, None)
    check_pages(model, ref, table, kv_lens)
    info = m.smla_cache_compact(pool, page, ref, table)       # in place
    assert info.cpu().tolist() == [n, k]
    check_pages(moved, ref, table, kv_lens)
    for s, d, r in model.copies + moved.copies:
        want[d, :r] = want[s, :r]
    assert np.array_equal(pool.cpu().numpy().reshape(want.shape), want)
    assert torch.equal(pool, keep)
    assert m.smla_device_status(clear=True) in ((0, -11) if num_pages < 10 else (0,))   # the tiny pool may run out


@pytest.mark.parametrize("used", [0, 1, 700])
def test_compact_of_empty_single_and_full_pools(used):
    num_pages, page = 700, 2
    ref = np.zeros(num_pages, np.int32)
    where = [] if used == 0 else [699] if used == 1 else range(700)
    ref[list(where)] = 3
    table = np.array([list(where)[:4] + [-1] * (4 - min(4, used))], np.int32)
    pool = torch.randint(0, 256, (num_pages * page, 600), device="cuda", dtype=torch.uint8)
    before = pool.cpu().numpy().copy()
    model = PageModel(ref, table, [0], page)
    n, k = model.compact()
    r, t = dev(ref), dev(table)
    info = m.smla_cache_compact(pool, page, r, t)
    assert info.cpu().tolist() == [n, k]
    check_pages(model, r, t, None)
    if used == 1:
        before[0:2, :ROW] = before[1398:1400, :ROW]           # the bytes between rows stay
    assert np.array_equal(pool.cpu().numpy(), before)


def test_pool_exhausted():
    page, num_pages = 4, 6
    ref, table, lens = _state(num_pages, page, 5, 4, [7, 6, 0, 0, 0], 4)      # 4 pages taken
    r, t, l = dev(ref), dev(table), dev(lens)
    pool = random_pool(num_pages, page, 4)
    m.smla_device_status(clear=True)
    m.smla_cache_fork(pool, page, r, t, l, dev(np.array([0, 1, 0], np.int32)), dev(np.array([2, 3, 4], np.int32)))
    assert m.smla_device_status(clear=True) == -11
    assert l.cpu().tolist() == [7, 6, 7, 6, 0] and t[4].cpu().tolist() == [-1] * 4
    assert (r > 0).all()
    m.smla_cache_reserve(page, r, t, dev(np.array([7, 6, 7, 6, 16], np.int32)))
    assert m.smla_device_status(clear=True) == -11
    assert t[4].cpu().tolist() == [-1] * 4
    m.smla_cache_free(r, t, l, dev(np.array([2, 2, 3, 2], np.int32)))          # the same row twice counts once
    assert m.smla_device_status(clear=True) == 0
    assert r.cpu().tolist() == list(ref)
    m.smla_cache_reserve(page, r, t, dev(np.array([7, 6, 0, 0, 16], np.int32)))  # two of four found
    assert m.smla_device_status(clear=True) == -11
    free = [p for p in range(num_pages) if ref[p] == 0]
    assert t[4].cpu().tolist() == free + [-1, -1]


def test_bad_ids_are_skipped_and_reported():
    page, num_pages = 4, 20
    ref, table, lens = _state(num_pages, page, 4, 5, [7, 20, 0, 0], 6)
    r, t, l = dev(ref), dev(table), dev(lens)
    pool = random_pool(num_pages, page, 6)
    before = pool.clone()

    def ints(*v):
        return dev(np.array(v, np.int32))

    def unchanged(code):
        assert m.smla_device_status(clear=True) == code
        assert r.cpu().tolist() == list(ref) and t.cpu().tolist() == table.tolist()
        assert l.cpu().tolist() == list(lens) and torch.equal(pool, before)

    m.smla_device_status(clear=True)
    m.smla_cache_free(r, t, l, ints(-1, 4))
    unchanged(-7)
    for p, c in ((-1, 2), (4, 2), (0, 4), (0, -3), (1, 1)):
        m.smla_cache_fork(pool, page, r, t, l, ints(p), ints(c))
        unchanged(-7)
    m.smla_cache_reserve(page, r, t, ints(7, 21, 0, -5))       # 21: past the table, which is mapped in full
    unchanged(-7)
    m.smla_cache_free(r, t, l, ints())
    m.smla_cache_fork(pool, page, r, t, l, ints(), ints())
    unchanged(0)
    l2 = ints(7, 21, 0, 0)                                      # a length past the table
    m.smla_cache_fork(pool, page, r, t, l2, ints(1), ints(2))
    unchanged(-7)
    t2 = t.clone()
    t2[2, 0] = num_pages                                        # a page id past the pool
    t2[3, 0] = int(np.flatnonzero(ref == 0)[-1])                # a page that nobody owns
    l2 = ints(7, 20, 4, 4)
    m.smla_cache_free(r, t2, l2, ints(2, 3))
    unchanged(-7)
    assert t2[2:].cpu().tolist() == [[-1] * 5] * 2


def test_page_calls_replayed_from_a_graph_follow_the_state():
    page, num_pages, R = 16, 300, 12
    ref, table, lens = _state(num_pages, page, R, 9, [100, 90] + [0] * 10, 8)
    pool = random_pool(num_pages, page, 8)
    r, t, l = dev(ref), dev(table), dev(lens)
    parents, children = dev(np.array([0, 1, 0], np.int32)), dev(np.array([4, 7, 9], np.int32))
    target = dev(np.zeros(R, np.int32))
    p = m.make_cache_params(num_pages, page, R, 9)
    ws = torch.empty(m.smla_cache_workspace_size(p), dtype=torch.uint8, device="cuda")

    def step():
        m.smla_cache_free(r, t, l, children)
        m.smla_cache_fork(pool, page, r, t, l, parents, children, workspace=ws)
        m.smla_cache_reserve(page, r, t, target, workspace=ws)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    model = PageModel(r.cpu(), t.cpu(), l.cpu(), page)
    for pr, ch, tg in (([1, 1, 0], [4, 7, 9], 33), ([0, 0, 0], [10, 11, 4], 140), ([1, 0, 1], [11, 9, 7], 1)):
        parents.copy_(dev(np.array(pr, np.int32)))
        children.copy_(dev(np.array(ch, np.int32)))
        target.fill_(tg)
        g.replay()
        model.free(ch)
        model.fork(pr, ch)
        model.reserve([tg] * R)
        check_pages(model, r, t, l)


def test_a_row_listed_twice_and_calls_on_a_side_stream():
    page, num_pages = 8, 64
    ref, table, lens = _state(num_pages, page, 5, 4, [30, 17, 8, 0, 0], 12)
    s = torch.cuda.Stream()
    r, t, l = dev(ref), dev(table), dev(lens)
    pool = random_pool(num_pages, page, 12)
    want = pool.cpu().numpy().copy()
    model = PageModel(ref, table, lens, page)
    s.wait_stream(torch.cuda.current_stream())
    m.smla_cache_free(r, t, l, dev(np.array([2, 2, 2], np.int32)), stream=s)
    model.free([2])
    m.smla_cache_fork(pool, page, r, t, l, dev(np.array([0, 0], np.int32)), dev(np.array([3, 4], np.int32)), stream=s)
    model.fork([0, 0], [3, 4])
    m.smla_cache_reserve(page, r, t, dev(np.array([32, 17, 9, 32, 31], np.int32)), stream=s)
    model.reserve([32, 17, 9, 32, 31])
    m.smla_cache_compact(pool, page, r, t, stream=s)
    model.compact()
    s.synchronize()
    check_pages(model, r, t, l)
    for a, b, rows in model.copies:
        want[b * page:b * page + rows] = want[a * page:a * page + rows]
    assert np.array_equal(pool.cpu().numpy(), want)


@pytest.mark.parametrize("stride,lead", [(ROW, 8), (600, 0), (1024, 16)])
def test_compact_of_strided_and_odd_pools(stride, lead):
    """Pages that start 8 bytes off a 16-byte boundary, and bytes between rows that stay."""
    page, num_pages = 7, 60
    pool = random_pool(num_pages, page, 14, stride, lead)
    before = pool.cpu().numpy().copy()
    rng = np.random.default_rng(14)
    ref = (rng.random(num_pages) < 0.5).astype(np.int32)
    table = np.flatnonzero(ref).astype(np.int32)[None, :].copy()
    model = PageModel(ref, table, [0], page)
    n, k = model.compact()
    r, t = dev(ref), dev(table)
    assert m.smla_cache_compact(pool, page, r, t).cpu().tolist() == [n, k]
    check_pages(model, r, t, None)
    for s, d, _ in model.copies:
        before[d * page:(d + 1) * page, :ROW] = before[s * page:(s + 1) * page, :ROW]
    assert np.array_equal(pool.cpu().numpy(), before)


def test_fork_of_a_parent_whose_last_page_is_not_mapped():
    page = 8
    pool = random_pool(6, page, 40)
    before = pool.clone()
    # parents: an unmapped last page (and a hole), a page past the pool, an ordinary one
    table = dev(np.array([[2, -1, -1], [4, 99, -1], [3, 5, -1], [-1] * 3, [-1] * 3, [-1] * 3], dtype=np.int32))
    lens = dev(np.array([19, 11, 12, 0, 0, 0], dtype=np.int32))
    ref = dev(np.array([0, 0, 1, 1, 1, 1], dtype=np.int32))
    m.smla_cache_fork(pool, page, ref, table, lens, dev(np.array([0, 1, 2], dtype=np.int32)),
                      dev(np.array([3, 4, 5], dtype=np.int32)))
    assert m.smla_device_status(clear=True) == -7     # page 99
    assert table.cpu().tolist()[3:] == [[2, -1, -1], [4, 99, -1], [3, 0, -1]]
    assert lens.cpu().tolist()[3:] == [19, 11, 12]
    assert ref.cpu().tolist() == [1, 0, 2, 2, 2, 1]               # one page taken, for the ordinary one
    assert torch.equal(pool[:4, :ROW], before[5 * page:5 * page + 4, :ROW])
    assert torch.equal(pool[4:], before[4:])
