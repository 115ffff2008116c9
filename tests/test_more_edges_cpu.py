"""Calls that need no GPU to be refused: pools whose rows cannot be what their distance says."""
import os
import subprocess
import sys

import pytest
import torch

import sparse_mla_decode_03_gb300 as m

from test_cache_cpu import lib  # noqa: F401


def _pools():
    wide = torch.zeros(32, 592, dtype=torch.uint8)
    return {
        "4-bit rows in 592-byte records": wide[:, :368],
        "the 8-bit rows' first 500 bytes": wide[:, :500],
        "4-bit rows in 584-byte records, one row": torch.zeros(1, 584, dtype=torch.uint8)[:, :360],
        "8-bit rows less than 584 bytes apart": torch.zeros(32 * 592, dtype=torch.uint8).as_strided((20, 584), (512, 1)),
        "rows wider than their distance": torch.zeros(32 * 592, dtype=torch.uint8).as_strided((20, 400), (368, 1)),
        "4-bit rows that are cut": torch.zeros(32, 368, dtype=torch.uint8)[:, :352],
    }


@pytest.mark.parametrize("what", list(_pools()))
def test_pools_whose_rows_are_not_what_their_distance_says(what):
    """Refused by every call that takes a pool, before it is told that the tensors are not on a GPU."""
    pool = _pools()[what]
    i1, i2 = torch.zeros(3, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    q, kv = torch.zeros(2, 64, 512, dtype=torch.bfloat16), torch.zeros(5, 512, dtype=torch.bfloat16)
    for call in (lambda: m.sparse_mla_decode(q, pool, i2),
                 lambda: m.sparse_mla_decode_paged(q, pool, i2, 1, i2),
                 lambda: m.sparse_mla_decode_split(q, pool, i2, 1),
                 lambda: m.sparse_mla_decode_noalloc(q, pool, i2),
                 lambda: m.sparse_mla_decode_simt(q, pool, i2),
                 lambda: m.smla_chunk_attention(q, pool, i2, 1, i1, i1[:2]),
                 lambda: m.smla_cache_append(kv, pool, i2, 1, i1, i1[:2]),
                 lambda: m.smla_cache_append_rotary(kv, pool, i2, 1, i1, i1[:2], torch.zeros(8, 64)),
                 lambda: m.smla_cache_read(pool, i2, 1, i1, i1[:2], 5),
                 lambda: m.smla_cache_fork(pool, 1, i1, i2, i1[:2], i1[:1], i1[:1]),
                 lambda: m.smla_cache_compact(pool, 1, i1, i2),
                 lambda: m.smla_cache_reorder(pool, 1, i1, i2, i1[:2], i1[:2])):
        with pytest.raises(ValueError, match="rows must hold"):
            call()


def test_pools_of_one_row():
    """A single row has no distance to another: its width tells what it is."""
    from sparse_mla_decode_03_gb300 import api
    q, i2 = torch.zeros(2, 64, 512, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32)
    for pool, stride in ((torch.zeros(4, 592, dtype=torch.uint8)[:1, :368], 368), (torch.zeros(1, 584, dtype=torch.uint8), 584),
                         (torch.zeros(4, 1024, dtype=torch.uint8)[:1], 584),
                         (torch.zeros(2000, dtype=torch.uint8).as_strided((1, 584), (16, 1)), 584)):
        with pytest.raises(ValueError, match="CUDA"):
            api._params_from(q, pool, i2, 1.0)
        assert api._check_rows("pool", pool) == stride


@pytest.mark.parametrize("stride,splits", [(368, 0), (584, 2)])
def test_no_place_for_a_workspace_size(lib, stride, splits):  # noqa: F811
    """A null pointer for the bytes is an error of the argument (in a process of its own)."""
    code = f"""
from ctypes import byref
import sparse_mla_decode_03_gb300 as m
from sparse_mla_decode_03_gb300 import _lib
p = byref(m.make_params(2, 64, 128, 1000, {stride}))
assert _lib.load().smla_paged_workspace_size(p, {splits}, None) == _lib.SMLA_ERR_INVALID_ARG"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    assert subprocess.run([sys.executable, "-c", code], cwd=root).returncode == 0
