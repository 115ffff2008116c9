"""Chunk attention on single SMs whose shares go from tiles of few rows to full ones and back: warps
without rows in one tile have some in the next.  Tolerances: _cache_helpers."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_03_gb300 as m

from _cache_helpers import SCALE, check_chunk, chunk_reference, dev, random_pool, tables
from _rows4_helpers import chunk_reference4, random_pool4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("H,kinds", [(16, (1, 4)), (16, (3, 1, 8)), (32, (1, 2)), (32, (3, 1))])
def test_tiles_of_few_rows_before_full_ones(bits, H, kinds):
    B, page = 420, 32
    rng = np.random.default_rng(H + len(kinds))
    ns = np.array([kinds[b % len(kinds)] for b in range(B)])
    lens = rng.integers(10, 190, B).astype(np.int32)
    num_pages = int(sum(-(-L // page) for L in lens)) + 2
    pool = (random_pool if bits == 8 else random_pool4)(num_pages, page, H)
    table = tables(lens, page, num_pages, H)
    cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    q = torch.randn(int(cu[-1]), H, 512, generator=torch.Generator().manual_seed(H)).to(torch.bfloat16).cuda()
    m.smla_device_status(clear=True)
    got = [m.smla_chunk_attention(q, pool, dev(table), page, dev(cu), dev(lens), softmax_scale=SCALE) for _ in range(4)]
    assert m.smla_device_status(clear=True) == 0
    check_chunk(got[0], (chunk_reference if bits == 8 else chunk_reference4)(q, pool, table, page, cu, lens))
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
