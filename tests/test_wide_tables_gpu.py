"""Page calls over tables whose rows have nearly 2^31 entries, the most that their width can say: the
count of a row's entries goes past an int behind the last ones."""
import pytest
import torch

import sparse_mla_decode_03_gb300 as m

from _cache_helpers import ROW

pytestmark = pytest.mark.gpu
WIDE = 2 ** 31 - 1


def _state(rows):
    """Rows of -7 (unmapped) with the last pages of the pool at both ends, which nothing else names."""
    if torch.cuda.mem_get_info()[0] < 10 * rows * WIDE:
        pytest.skip("not enough memory")
    pool = torch.arange(16 * ROW, device="cuda").to(torch.uint8).view(16, ROW)
    ref = torch.zeros(8, dtype=torch.int32, device="cuda")
    table = torch.full((rows, WIDE), -7, dtype=torch.int32, device="cuda")
    for r in range(rows):
        table[r, 0], table[r, 1], table[r, -1] = 7 - 3 * r, 6 - 3 * r, 5 - 3 * r
        ref[5 - 3 * r:8 - 3 * r] = 1
    return pool, ref, table, torch.full((rows,), 3, dtype=torch.int32, device="cuda")


def _rest(row, n):
    return bool((row[n:] == -1).all())


def test_reorder_empties_a_row():
    pool, ref, table, lens = _state(1)
    m.smla_device_status(clear=True)
    m.smla_cache_reorder(pool, 2, ref, table, lens, torch.full((1,), -1, dtype=torch.int32, device="cuda"))
    assert m.smla_device_status(clear=True) == 0
    assert not ref.any() and lens.item() == 0 and _rest(table[0], 0)


@pytest.mark.parametrize("call", ["reorder", "fork"])
def test_a_row_becomes_a_copy(call):
    """Row 0 goes on from row 1: one full page of it shared, one copied, nothing behind."""
    pool, ref, table, lens = _state(2)
    m.smla_device_status(clear=True)
    if call == "reorder":        # row 1 has two children, of which row 0 takes it over; row 1 shares
        m.smla_cache_reorder(pool, 2, ref, table, lens, torch.ones(2, dtype=torch.int32, device="cuda"))
    else:
        m.smla_cache_fork(pool, 2, ref, table, lens, *torch.tensor([[1], [0]], dtype=torch.int32, device="cuda"))
    assert m.smla_device_status(clear=True) == 0
    assert lens.tolist() == [3, 3]
    taker, sharer = (0, 1) if call == "reorder" else (1, 0)
    assert table[taker, [0, 1, 2, -2, -1]].tolist() == [4, 3, -7, -7, 2]
    assert bool((table[taker, 2:-1] == -7).all())
    assert table[sharer, :2].tolist() == [4, 0] and _rest(table[sharer], 2)
    counts = [1, 0, 1, 1, 2, 0, 0, 0] if call == "reorder" else [1, 0, 1, 1, 2, 1, 1, 1]
    assert ref.tolist() == counts
    assert torch.equal(pool[0], pool[6])


def test_free_empties_a_row():
    pool, ref, table, lens = _state(1)
    m.smla_device_status(clear=True)
    m.smla_cache_free(ref, table, lens, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert m.smla_device_status(clear=True) == 0
    assert not ref.any() and lens.item() == 0
    # entries that are unmapped stay what they are
    assert table[0, [0, 1, 2, -2, -1]].tolist() == [-1, -1, -7, -7, -1]
