"""Refusals of the paged-cache calls at the edges of their sizes."""
import ctypes

import pytest

import sparse_mla_decode_03_gb300 as m
from sparse_mla_decode_03_gb300 import _lib

from test_cache_cpu import P, lib, vp  # noqa: F401


@pytest.mark.parametrize("seqs,width,refused", [(65535, 32769, True), (2, 1 << 30, True), (1, 2 ** 31 - 1, False),
                                                (65535, 32768, False)])
def test_reserve_over_tables_whose_entries_pass_an_int(lib, seqs, width, refused):  # noqa: F811
    """Entries that want a page are counted in ints: a table of 2^31 and more is refused, before any
    other check that a call without a GPU or a workspace fails."""
    c = m.make_cache_params(100, 16, seqs, width)
    st = lib.smla_cache_reserve(P, P, P, ctypes.byref(c), P, 0, vp(0))
    assert st == (_lib.SMLA_ERR_UNSUPPORTED_SHAPE if refused else _lib.SMLA_ERR_WORKSPACE_TOO_SMALL)
