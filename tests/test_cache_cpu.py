"""Refusals of the paged-cache and chunk-attention entry points that need no GPU."""
import ctypes
import os

import pytest
import torch

import sparse_mla_decode_03_gb300 as m
from sparse_mla_decode_03_gb300 import _lib

vp = ctypes.c_void_p
P = vp(4096)          # an aligned address that is never read: the calls are refused before that
INV, SHAPE, WS = _lib.SMLA_ERR_INVALID_ARG, _lib.SMLA_ERR_UNSUPPORTED_SHAPE, _lib.SMLA_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from sparse_mla_decode_03_gb300 import build
        build.build()
    return _lib.load()


def _cache(**over):
    c = m.make_cache_params(100, 16, 4, 8)
    for k, v in over.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def _chunk(**over):
    p = m.make_chunk_params(2, 64, 10, 16, 8, 1600, 584, 256)
    for k, v in over.items():
        setattr(p, k, v)
    return ctypes.byref(p)


@pytest.mark.parametrize("over,code", [
    ({"num_pages": 0}, INV), ({"page_size": 0}, INV), ({"num_seqs": 0}, INV), ({"max_pages": 0}, INV),
    ({"kv_row_stride": 583}, INV), ({"kv_row_stride": 588}, INV), ({"num_seqs": 65536}, SHAPE),
    ({"num_pages": 1 << 30, "page_size": 4}, SHAPE),
])
def test_cache_params(lib, over, code):
    n = ctypes.c_size_t()
    c = _cache(**over)
    assert lib.smla_cache_workspace_size(c, ctypes.byref(n)) == code
    assert lib.smla_cache_append(P, 512, 1, P, P, P, P, c, vp(0)) == code
    assert lib.smla_cache_reserve(P, P, P, c, P, 1 << 30, vp(0)) == code
    assert lib.smla_cache_fork(P, P, P, P, P, P, 1, c, P, 1 << 30, vp(0)) == code
    assert lib.smla_cache_free(P, P, P, P, 1, c, vp(0)) == code
    assert lib.smla_cache_compact(P, P, P, P, P, P, c, P, 1 << 30, vp(0)) == code


def test_cache_pointers(lib):
    c = _cache()
    n = ctypes.c_size_t()
    assert lib.smla_cache_workspace_size(c, ctypes.byref(n)) == 0
    assert lib.smla_cache_workspace_size(None, ctypes.byref(n)) == INV
    assert lib.smla_cache_workspace_size(c, None) == INV

    def each(call, count, skip=()):
        for i in range(count):
            if i not in skip:
                for bad in (vp(0), vp(4097)):
                    args = [P] * count
                    args[i] = bad
                    assert call(*args) == INV, i

    each(lambda kv, pool, t, cu, l: lib.smla_cache_append(kv, 512, 1, pool, t, cu, l, c, vp(0)), 5)
    each(lambda r, t, l, w: lib.smla_cache_reserve(r, t, l, c, w, n, vp(0)), 4)
    each(lambda k, r, t, l, p, ch, w: lib.smla_cache_fork(k, r, t, l, p, ch, 1, c, w, n, vp(0)), 7)
    each(lambda r, t, l, x: lib.smla_cache_free(r, t, l, x, 1, c, vp(0)), 4)
    each(lambda k, r, t, ro, to, i, w: lib.smla_cache_compact(k, r, t, ro, to, i, c, w, n, vp(0)), 7)
    assert lib.smla_cache_append(P, 511, 1, P, P, P, P, c, vp(0)) == INV
    assert lib.smla_cache_append(P, 516, 1, P, P, P, P, c, vp(0)) == INV
    assert lib.smla_cache_append(P, 512, -1, P, P, P, P, c, vp(0)) == INV
    assert lib.smla_cache_append(vp(0), 512, 0, P, P, P, P, c, vp(0)) == 0       # nothing to write
    assert lib.smla_cache_free(P, P, P, vp(0), 0, c, vp(0)) == 0
    assert lib.smla_cache_free(P, P, P, P, -1, c, vp(0)) == INV
    assert lib.smla_cache_fork(P, P, P, P, vp(0), vp(0), 0, c, P, n, vp(0)) == 0
    assert lib.smla_cache_fork(P, P, P, P, P, P, 5, c, P, n, vp(0)) == INV       # more than num_seqs
    short = n.value - 1
    assert lib.smla_cache_reserve(P, P, P, c, P, short, vp(0)) == WS
    assert lib.smla_cache_fork(P, P, P, P, P, P, 1, c, P, short, vp(0)) == WS
    assert lib.smla_cache_compact(P, P, P, P, P, P, c, P, short, vp(0)) == WS


@pytest.mark.parametrize("over,code", [
    ({"batch": 0}, INV), ({"batch": 65536}, SHAPE), ({"num_heads": 8}, SHAPE), ({"num_heads": 48}, SHAPE),
    ({"total_q": 0}, INV), ({"total_q": 1 << 24}, SHAPE), ({"page_size": 0}, INV), ({"max_pages": 0}, INV),
    ({"reserved": 1}, INV), ({"num_rows": 0}, INV), ({"kv_row_stride": 576}, INV), ({"kv_row_stride": 590}, INV),
    ({"max_kv_tokens": 0}, INV), ({"softmax_scale": 0.0}, INV), ({"softmax_scale": float("nan")}, INV),
    ({"num_rows": (1 << 31) + 1}, SHAPE), ({"kv_row_stride": 1 << 31}, SHAPE), ({"max_kv_tokens": (1 << 30) + 1}, SHAPE),
    ({"logit_cap": -1.0}, INV), ({"logit_cap": float("inf")}, INV),
])
def test_chunk_params(lib, over, code):
    n = ctypes.c_size_t()
    p = _chunk(**over)
    assert lib.smla_chunk_workspace_size(p, ctypes.byref(n)) == code
    assert lib.smla_chunk_attention(P, P, P, P, P, vp(0), vp(0), vp(0), P, P, p, P, 1 << 40, vp(0)) == code


def test_chunk_pointers(lib):
    for i in (0, 1, 2, 3, 4, 8, 9, 11):
        for bad in (vp(0), vp(4097)):
            args = [P] * 10 + [_chunk(), P, 1 << 40, vp(0)]
            args[i] = bad
            assert lib.smla_chunk_attention(*args) == INV, i
    for i in (5, 6, 7):                     # optional, but aligned
        args = [P] * 10 + [_chunk(), P, 1 << 40, vp(0)]
        args[i] = vp(4098)
        assert lib.smla_chunk_attention(*args) == INV, i


def test_binding_checks():
    pool = torch.zeros(32, 584, dtype=torch.uint8)
    i1, i2 = torch.zeros(3, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    kv = torch.zeros(5, 512, dtype=torch.bfloat16)
    for call in (lambda: m.smla_cache_append(kv, pool, i2, 16, i1, i1[:2]),              # not on a GPU
                 lambda: m.smla_cache_append(kv, pool[:, :583], i2, 16, i1, i1[:2]),
                 lambda: m.smla_cache_append(kv, pool.int(), i2, 16, i1, i1[:2]),
                 lambda: m.smla_cache_append(kv, pool, i2, 33, i1, i1[:2]),
                 lambda: m.smla_cache_reserve(16, i1, i2, i1),
                 lambda: m.smla_cache_free(i1, i2, i1, i1),
                 lambda: m.smla_cache_fork(pool, 16, i1, i2, i1, i1, i1),
                 lambda: m.smla_cache_compact(pool, 16, i1, i2),
                 lambda: m.smla_chunk_attention(torch.zeros(5, 64, 512, dtype=torch.bfloat16), pool, i2, 16, i1,
                                                i1[:2])):
        with pytest.raises(ValueError):
            call()


def test_chunk_workspace_of_single_tokens_holds_no_copy_of_the_cache(lib):
    def need(**over):
        n = ctypes.c_size_t()
        assert lib.smla_chunk_workspace_size(_chunk(**over), ctypes.byref(n)) == 0
        return n.value

    few = dict(batch=4, num_heads=64, total_q=15)           # 240 rows a sequence on average
    many = dict(batch=4, num_heads=64, total_q=16)
    assert need(**few, max_kv_tokens=1 << 30) == need(**few, max_kv_tokens=1)
    assert need(**many, max_kv_tokens=65 * 64) - need(**many, max_kv_tokens=64) == 64 * (64 * 1024 + 16)
