"""The paged cache's calls at the edges of what their arguments allow."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_03_gb300 as m

from _cache_helpers import PageModel, check_pages, dev, random_pool

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
