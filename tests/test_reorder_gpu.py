"""smla_cache_reorder against its definition on lists: counts, tables, lengths and rows exactly."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_03_gb300 as m

from _cache_helpers import PageModel, ROW, check_pages, dev, tables
from _rows4_helpers import ROW4, reorder_model

pytestmark = pytest.mark.gpu


def _ints(v):
    return dev(np.asarray(v, np.int32))


def _state(lens, page, num_pages, seed, row=ROW, stride=None, extra=2):
    stride = stride or row
    g = torch.Generator().manual_seed(seed)
    pool = torch.randint(0, 256, (num_pages * page, stride), generator=g, dtype=torch.uint8).cuda()
    table = tables(lens, page, num_pages, seed, extra)
    ref = np.zeros(num_pages, np.int32)
    ref[table[table >= 0]] = 1
    return pool, ref, table, np.array(lens, np.int32)


def _check(pool, ref, table, lens, page, parents, row=ROW, status=0, times=1, **kw):
    model = PageModel(ref, table, lens, page)
    want = pool.cpu().numpy().copy()
    r, t, l, p = dev(ref), dev(table), dev(lens), _ints(parents)
    for _ in range(times):
        m.smla_device_status(clear=True)
        m.smla_cache_reorder(pool, page, r, t, l, p, **kw)
        assert m.smla_device_status(clear=True) == status
        model.copies = []
        reorder_model(model, parents)
        check_pages(model, r, t, l)
        rows = want.copy()
        for a, b, k in model.copies:
            rows[b * page:b * page + k, :row] = want[a * page:a * page + k, :row]
        want = rows
        assert np.array_equal(pool.cpu().numpy(), want)
    return r, t, l


@pytest.mark.parametrize("row,stride", [(ROW, ROW), (ROW, 600), (ROW4, ROW4), (ROW4, 400)])
@pytest.mark.parametrize("page", [1, 16, 100])
def test_random_parents(row, stride, page):
    rng = np.random.default_rng(page + stride)
    lens = [int(v) for v in rng.integers(0, 400, 24)]
    lens[3] = 3 * page
    pages = sum(-(-L // page) for L in lens) + 40
    state = _state(lens, page, pages, page, row, stride)
    parents = rng.integers(0, 24, 24)
    _check(*state, page, parents, row, times=3)


def test_identity_and_permutation_move_nothing():
    lens, page = [33, 0, 64, 17, 1], 16
    pool, ref, table, lens = _state(lens, page, 20, 1)
    before = pool.clone()
    r, t, l = _check(pool, ref, table, lens, page, range(5))
    assert torch.equal(t.cpu(), torch.as_tensor(table)) and torch.equal(r.cpu(), torch.as_tensor(ref))
    _check(pool, ref, table, lens, page, [4, 2, 0, 1, 3])
    assert torch.equal(pool, before)


def test_rows_to_be_emptied_and_bad_parents():
    pool, ref, table, lens = _state([20, 40, 7, 33], 16, 20, 2)
    _check(pool, ref, table, lens, 16, [-1, 1, -5, 1])
    _check(pool, ref, table, lens, 16, [4, 1, 2 ** 31 - 1, -2 ** 31], status=-7)
    _check(pool, ref, table, lens, 16, [-1] * 4)


def test_a_dropped_row_makes_room_for_a_copy():
    """No page is free but those of the row that nobody goes on from."""
    page = 16
    pool, ref, table, lens = _state([20, 24], page, 4, 3, extra=1)
    assert (ref == 1).all()
    _check(pool, ref, table, lens, page, [0, 0])
    pool, ref, table, lens = _state([24, 5], page, 3, 4, extra=1)
    _check(pool, ref, table, lens, page, [1, 1])


def test_an_exhausted_pool_leaves_a_child_empty():
    pool, ref, table, lens = _state([20, 16, 24], 16, 5, 5)
    _check(pool, ref, table, lens, 16, [0, 0, 0], times=1)
    pool, ref, table, lens = _state([20, 0, 0, 24], 16, 4, 6)
    _check(pool, ref, table, lens, 16, [0, 0, 0, 3], status=-11)


def test_reserved_pages_stay_with_the_lowest_child():
    page = 16
    pool, ref, table, lens = _state([20, 20], page, 12, 7, extra=4)
    free = [p for p in range(12) if ref[p] == 0]
    table[0, 2], table[0, 4] = free[0], free[1]
    ref[free[:2]] = 1
    r, t, _ = _check(pool, ref, table, lens, page, [0, 0])
    assert t[0, 2] == free[0] and t[1, 2] == -1
    _check(pool, ref, table, lens, page, [1, 0])
    _check(pool, ref, table, lens, page, [1, 1])


def test_lengths_and_entries_that_are_wrong():
    page = 16
    pool, ref, table, lens = _state([20, 30, 40], page, 12, 8, extra=0)
    lens[0], lens[1] = 1000, -4          # cut to the table; no tokens
    _check(pool, ref, table, lens, page, [0, 0, 1], status=-7)
    pool, ref, table, lens = _state([40, 30, 40], page, 12, 9)
    table[0, 1], table[2, 0] = -1, 12    # unmapped; past the pool
    _check(pool, ref, table, lens, page, [0, 0, 1], status=-7)
    _check(pool, ref, table, lens, page, [2, 2, 0], status=-7)
    table[2, 0] = 0
    table[0, 2] = -1                     # the last page is not mapped: nothing to copy
    ref[:] = 0
    ref[table[table >= 0]] = 1
    _check(pool, ref, table, lens, page, [0, 0, 2])


def test_many_rows_and_a_wide_table():
    rng = np.random.default_rng(11)
    lens = [int(v) for v in rng.integers(0, 9, 9000)]
    pages = sum(-(-L // 4) for L in lens) + 5000
    _check(*_state(lens, 4, pages, 11, ROW4), 4, rng.integers(-1, 9000, 9000), ROW4)
    lens = [3001, 12, 5000]
    _check(*_state(lens, 1, 8200, 12, ROW4, extra=70000), 1, [2, 2, 0], ROW4)


def test_replay_on_a_side_stream():
    page = 16
    pool, ref, table, lens = _state([50, 60, 70, 33], page, 40, 13)
    r, t, l, p = dev(ref), dev(table), dev(lens), _ints([0, 1, 2, 3])
    ws = torch.empty(m.smla_cache_reorder_workspace_size(m.make_cache_params(40, page, 4, table.shape[1])),
                     dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    m.smla_cache_reorder(pool, page, r, t, l, p, workspace=ws, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        m.smla_cache_reorder(pool, page, r, t, l, p, workspace=ws, stream=s)
    model = PageModel(ref, table, lens, page)
    for parents in ([1, 1, 0, 3], [3, 3, 3, 3], [2, 0, 1, -1]):
        p.copy_(_ints(parents))
        g.replay()
        torch.cuda.synchronize()
        reorder_model(model, parents)
        check_pages(model, r, t, l)
