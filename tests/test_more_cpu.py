"""Refusals that need no GPU: rows of 4-bit values, the append with a rotation, reading back,
reordering, selection over beams."""
import ctypes
import os

import pytest
import torch

import sparse_mla_decode_03_gb300 as m
from sparse_mla_decode_03_gb300 import _lib

vp = ctypes.c_void_p
P = vp(4096)          # an aligned address that is never read: the calls are refused before that
INV, SHAPE, WS = _lib.SMLA_ERR_INVALID_ARG, _lib.SMLA_ERR_UNSUPPORTED_SHAPE, _lib.SMLA_ERR_WORKSPACE_TOO_SMALL
n = ctypes.c_size_t()


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from sparse_mla_decode_03_gb300 import build
        build.build()
    return _lib.load()


def _with(p, **over):
    for k, v in over.items():
        setattr(p, k, v)
    return ctypes.byref(p)


def _cache(**over):
    return _with(m.make_cache_params(100, 16, 4, 8), **over)


def _rotary(**over):
    return _with(_lib.SmlaRotaryParams(4096, 4096, 4096, 100, 1024, 64, 8192, 512, 16, 0, 0), **over)


def _beam(**over):
    return _with(m.make_beam_params(3, 4, 1000, 8), **over)


@pytest.mark.parametrize("stride", [0, -16, 8, 360, 364, 376, 511, 528, 576, 583, 588])
def test_row_strides_that_hold_no_rows(lib, stride):
    c = _cache(kv_row_stride=stride)
    assert lib.smla_cache_workspace_size(c, ctypes.byref(n)) == INV
    assert lib.smla_cache_reorder_workspace_size(c, ctypes.byref(n)) == INV
    assert lib.smla_cache_append(P, 512, 1, P, P, P, P, c, vp(0)) == INV
    assert lib.smla_cache_append_rotary(P, 512, 1, P, P, P, P, c, _rotary(), vp(0)) == INV
    assert lib.smla_cache_read(P, P, P, P, P, 512, 1, c, vp(0)) == INV
    assert lib.smla_cache_reorder(P, P, P, P, P, c, P, 1 << 30, vp(0)) == INV
    p = m.make_chunk_params(2, 64, 10, 16, 8, 1600, stride, 256)
    assert lib.smla_chunk_workspace_size(ctypes.byref(p), ctypes.byref(n)) == INV
    p = m.make_params(2, 64, 128, 1000, stride)
    assert lib.smla_workspace_size(ctypes.byref(p), 0, ctypes.byref(n)) == INV


@pytest.mark.parametrize("stride", [368, 384, 496, 512])
def test_row_strides_of_4_bit_values(lib, stride):
    assert lib.smla_cache_workspace_size(_cache(kv_row_stride=stride), ctypes.byref(n)) == 0
    p = m.make_chunk_params(2, 64, 10, 16, 8, 1600, stride, 256)
    assert lib.smla_chunk_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0
    p = ctypes.byref(m.make_params(2, 64, 128, 1000, stride))
    assert lib.smla_workspace_size(p, 0, ctypes.byref(n)) == 0
    need = n.value
    assert lib.smla_paged_workspace_size(p, 0, ctypes.byref(n)) == 0 and n.value == need
    assert lib.smla_workspace_size(p, 1, ctypes.byref(n)) == INV            # the split is not the caller's
    assert lib.sparse_mla_decode(P, P, P, P, P, p, 1, P, 1 << 40, vp(0)) == INV
    assert lib.sparse_mla_decode(P, P, P, P, P, p, 0, P, need - 1, vp(0)) == WS
    assert lib.sparse_mla_decode(P, P, P, P, P, p, 0, vp(4100), need, vp(0)) == INV
    assert lib.sparse_mla_decode_paged(P, P, P, 8, 16, P, P, P, p, 0, P, need - 1, vp(0)) == WS
    assert lib.sparse_mla_decode_paged(P, P, P, 8, 0, P, P, P, p, 0, P, need, vp(0)) == INV
    i = ctypes.c_int32()
    assert lib.smla_default_num_splits(p, ctypes.byref(i)) == SHAPE
    assert lib.smla_decode_plan(p, 0, ctypes.byref(i), ctypes.byref(i)) == SHAPE
    assert lib.sparse_mla_decode_split(P, P, P, p, 1, P, P, vp(0)) == SHAPE
    assert lib.sparse_mla_decode_simt(P, P, P, P, P, p, vp(0)) == SHAPE
    assert lib.sparse_mla_decode_noalloc(P, P, P, P, P, p, 0, vp(0)) == SHAPE
    assert lib.sparse_mla_decode_noalloc(P, P, P, P, P, p, 1, vp(0)) == INV
    # 16-byte pieces of rows: the pool starts on one
    c = _cache(kv_row_stride=stride)
    assert lib.smla_cache_append(P, 512, 1, vp(4104), P, P, P, c, vp(0)) == INV
    assert lib.smla_cache_reorder(vp(4104), P, P, P, P, c, P, 1 << 30, vp(0)) == INV


@pytest.mark.parametrize("over,code", [
    ({"table": 0}, INV), ({"table": 4100}, INV), ({"table_rows": 0}, INV), ({"num_heads": -1}, INV), ({"pairing": 2}, INV),
    ({"pairing": -1}, INV), ({"reserved": 1}, INV), ({"q": 0}, INV), ({"q_rope": 0}, INV), ({"q": 4104}, INV),
    ({"q_rope": 4104}, INV), ({"q_rope_token_stride": 4}, INV), ({"q_rope_head_stride": 63}, INV),
    ({"q_token_stride": -8}, INV), ({"q_head_stride": 513}, INV), ({"num_heads": 2 ** 31 - 1}, SHAPE),
])
def test_rotary_params(lib, over, code):
    assert lib.smla_cache_append_rotary(P, 512, 100, P, P, P, P, _cache(), _rotary(**over), vp(0)) == code


def test_token_calls(lib):
    c, r = _cache(), _rotary()
    for i in range(5):
        for bad in (vp(0), vp(4097)):
            a = [P] * 5
            a[i] = bad
            assert lib.smla_cache_append_rotary(a[0], 512, 1, *a[1:], c, r, vp(0)) == INV
            assert lib.smla_cache_read(*a, 512, 1, c, vp(0)) == INV
    assert lib.smla_cache_append_rotary(P, 512, 1, P, P, P, P, c, None, vp(0)) == INV
    for stride, total in ((511, 1), (516, 1), (512, -1)):
        assert lib.smla_cache_append_rotary(P, stride, total, P, P, P, P, c, r, vp(0)) == INV
        assert lib.smla_cache_read(P, P, P, P, P, stride, total, c, vp(0)) == INV
    # nothing to do
    assert lib.smla_cache_append_rotary(vp(0), 512, 0, P, P, P, P, c, _rotary(q=0, q_rope=0), vp(0)) == 0
    assert lib.smla_cache_read(P, P, P, P, vp(0), 512, 0, c, vp(0)) == 0
    assert lib.smla_cache_append_rotary(vp(0), 512, 0, P, P, P, P, c, _rotary(pairing=2), vp(0)) == INV


def test_reorder_pointers_and_workspace(lib):
    c = _cache()
    assert lib.smla_cache_reorder_workspace_size(c, ctypes.byref(n)) == 0
    assert n.value == 5 * 256                       # four lists of 4 rows, a table of 4 x 8
    assert lib.smla_cache_reorder_workspace_size(None, ctypes.byref(n)) == INV
    assert lib.smla_cache_reorder_workspace_size(c, None) == INV
    for i in range(6):
        for bad in (vp(0), vp(4097)):
            a = [P] * 6
            a[i] = bad
            assert lib.smla_cache_reorder(*a[:5], c, a[5], 1 << 30, vp(0)) == INV
    assert lib.smla_cache_reorder(P, P, P, P, P, c, P, 5 * 256 - 1, vp(0)) == WS


@pytest.mark.parametrize("over,code", [
    ({"groups": 0}, INV), ({"beams": 0}, INV), ({"vocab": 0}, INV), ({"num_out": 0}, INV), ({"num_out": -1}, INV),
    ({"row_stride": 999}, INV), ({"row_stride": -1}, INV), ({"logits_type": 3}, INV), ({"logits_type": -1}, INV),
    ({"reserved": 1}, INV), ({"beams": 65}, SHAPE), ({"num_out": 65}, SHAPE), ({"groups": 16384}, SHAPE),
    ({"vocab": (1 << 24) + 1, "row_stride": 1 << 25}, SHAPE), ({"row_stride": (1 << 40) + 1}, SHAPE),
])
def test_beam_params(lib, over, code):
    p = _beam(**over)
    assert lib.smla_beam_workspace_size(p, ctypes.byref(n)) == code
    assert lib.smla_beam_select(P, P, vp(0), P, P, P, p, P, 1 << 40, vp(0)) == code


def test_beam_pointers_and_workspace(lib):
    p = _beam()
    assert lib.smla_beam_workspace_size(p, ctypes.byref(n)) == 0
    assert lib.smla_beam_workspace_size(None, ctypes.byref(n)) == INV
    assert lib.smla_beam_workspace_size(p, None) == INV
    assert lib.smla_beam_select(P, P, vp(0), P, P, P, p, P, n.value - 1, vp(0)) == WS
    for i in (0, 1, 3, 4, 5, 6):
        for bad in (vp(0), vp(4097)):
            a = [P, P, vp(0), P, P, P, P]
            a[i] = bad
            assert lib.smla_beam_select(*a[:6], p, a[6], 1 << 40, vp(0)) == INV, i
    for end in (-1, 1000):                          # read with finished beams only
        assert lib.smla_beam_select(P, P, P, P, P, P, _beam(end_token=end), P, 1 << 40, vp(0)) == INV
        assert lib.smla_beam_select(P, P, vp(0), P, P, P, _beam(end_token=end), P, 0, vp(0)) == WS


def test_binding_checks():
    i1, i2 = torch.zeros(3, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    kv, q = torch.zeros(5, 512, dtype=torch.bfloat16), torch.zeros(2, 64, 512, dtype=torch.bfloat16)
    pool, turn = torch.zeros(32, 368, dtype=torch.uint8), torch.zeros(8, 64)
    wide = torch.zeros(32, 584, dtype=torch.uint8)
    for call in (lambda: m.smla_cache_append_rotary(kv, pool, i2, 16, i1, i1[:2], turn),            # not on a GPU
                 lambda: m.smla_cache_read(pool, i2, 16, i1, i1[:2], 5),
                 lambda: m.smla_cache_reorder(pool, 16, i1, i2, i1[:2], i1[:2]),
                 lambda: m.smla_beam_select(torch.zeros(4, 9), torch.zeros(2, 2)),
                 lambda: m.smla_beam_select(torch.zeros(4, 9, dtype=torch.int32), torch.zeros(2, 2)),
                 lambda: m.smla_cache_append(kv, pool[:, :360], i2, 16, i1, i1[:2]),
                 lambda: m.smla_cache_append(kv, wide[:, :368], i2, 16, i1, i1[:2]),                # 584 bytes apart
                 lambda: m.sparse_mla_decode(q, pool[:, :200], i2)):
        with pytest.raises(ValueError):
            call()
