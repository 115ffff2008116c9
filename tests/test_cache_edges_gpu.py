"""The paged cache's calls at the edges of what their arguments allow."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_03_gb300 as m

from _cache_helpers import PageModel, ROW, check_pages, dev, pack_rows, random_pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("num_pages", [8, 5000])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("stale", ["hole", "behind", "past the pool", None])
def test_compact_copies_and_reports_entries_that_name_no_page_in_use(num_pages, in_place, stale):
    """An entry that names a page nobody owns, below the pages in use (a hole, which then holds
    another page's rows) or behind them, or no page of the pool."""
    page = 2
    pool = random_pool(num_pages, page, 1)
    ref = np.zeros(num_pages, np.int32)
    ref[1::2] = 1                                   # half are in use, the odd ones
    width = num_pages // 2
    table = np.full((3, width), -1, np.int32)
    table[0] = np.arange(1, num_pages, 2)[::-1]
    table[2, :2] = (-3, 1)                          # any negative number is an unmapped entry
    ref[1] = 2
    if stale is not None:
        table[1, 1] = {"hole": 2, "behind": num_pages - 2, "past the pool": num_pages}[stale]
    model = PageModel(ref, table, [0, 0, 0], page)
    n, k = model.compact()
    if stale is not None:
        model.table[1][1] = int(table[1, 1])
    r, t = dev(ref), dev(table)
    outs = {} if in_place else {"ref_count_out": torch.full_like(r, -9), "block_table_out": torch.full_like(t, -9)}
    m.smla_device_status(clear=True)
    info = m.smla_cache_compact(pool, page, r, t, **outs)
    assert m.smla_device_status(clear=True) == (0 if stale is None else -7)
    assert info.cpu().tolist() == [n, k]
    check_pages(model, outs.get("ref_count_out", r), outs.get("block_table_out", t), None)


@pytest.mark.parametrize("bits,status", [(0x7F77, 0), (0x7F78, -8), (0x7F7F, -8), (0x7F60, 0), (0x7F61, 0)])
@pytest.mark.parametrize("sign", [0, 0x8000])
@pytest.mark.parametrize("col", [0, 63, 100, 447, 448, 511])
def test_append_reports_values_that_round_past_the_largest(bits, status, sign, col):
    """1.9375 * 2^127 (bf16 0x7f78) is halfway between 240 and 256 in the scale 2^120 and rounds to
    the even 256: 2^128.  A rope value is copied, and never out of range."""
    kv = torch.randn(3, 512, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    kv[1].view(torch.int16)[col] = (bits | sign) - (65536 if sign else 0)
    pool = torch.zeros((4, ROW), dtype=torch.uint8, device="cuda")
    m.smla_device_status(clear=True)
    m.smla_cache_append(kv.cuda(), pool, dev(np.zeros((1, 1), np.int32)), 4, dev(np.array([0, 3], np.int32)),
                        dev(np.array([3], np.int32)))
    assert m.smla_device_status(clear=True) == (status if col < 448 else 0)
    want = pack_rows(kv)
    assert np.array_equal(pool[:3].cpu().numpy(), want) and not pool[3].any()
    if col < 448:
        top = want[1, col] & 0x7F
        assert (top >= 0x78) == (status != 0) if want[1, 448 + col // 64] == 247 else status == 0


@pytest.mark.parametrize("short", [0, 6, 7, 2000])
def test_reserve_from_as_many_pages_as_an_int_counts(short):
    """2^31 - 1 pages: the parts of the counts that the blocks and threads of the plan take end
    next to the largest int."""
    n = 2 ** 31 - 1 - short
    ref = torch.ones(n, dtype=torch.int32, device="cuda")
    free = [5, 2 ** 28 + 1, 2 ** 30 + 7, n - 1030, n - 2, n - 1]
    ref[torch.tensor(free, device="cuda")] = 0
    table = dev(np.full((2, 4), -1, np.int32))
    m.smla_device_status(clear=True)
    m.smla_cache_reserve(1, ref, table, dev(np.array([3, 2], np.int32)))
    assert m.smla_device_status(clear=True) == 0
    assert table.cpu().tolist() == [free[:3] + [-1], free[3:5] + [-1, -1]]
    assert ref[-1].item() == 0 and ref[torch.tensor(free[:5], device="cuda")].tolist() == [1] * 5
    m.smla_cache_reserve(1, ref, table, dev(np.array([4, 3], np.int32)))
    assert m.smla_device_status(clear=True) == -11
    assert table.cpu().tolist() == [free[:3] + [free[5]], free[3:5] + [-1, -1]]
    assert int(ref.min()) == 1 and int(ref.max()) == 1
