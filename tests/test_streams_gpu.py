"""Calls of the binding with `stream=` another stream than the current one: what they allocate,
and what the caller drops right after the call, stays theirs until that stream has come to it.

The allocations are looked at with the library's entry points replaced by ones that note their
arguments and launch nothing."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_mla_decode_03_gb300 as m
from sparse_mla_decode_03_gb300 import _lib
from sparse_mla_decode_03_gb300 import workloads as W

from _cache_helpers import PageModel, ROW, SCALE, check_chunk, check_pages, chunk_reference, dev, random_pool, tables

pytestmark = pytest.mark.gpu

SIZES = ("smla_default_num_splits", "smla_decode_plan", "smla_workspace_size", "smla_paged_workspace_size",
         "smla_cache_workspace_size", "smla_chunk_workspace_size", "smla_status_string")


class NoLaunch:
    """The library with entry points that note the addresses they get and do nothing."""

    def __init__(self, lib):
        self.lib, self.seen = lib, []

    def __getattr__(self, name):
        if name in SIZES:
            return getattr(self.lib, name)

        def call(*args):
            self.seen = [v for v in (a.value if isinstance(a, ctypes.c_void_p) else a for a in args)
                         if isinstance(v, int) and v > 1 << 32]
            return 0
        return call


@pytest.fixture
def quiet(monkeypatch):
    fake = NoLaunch(_lib.load())
    monkeypatch.setattr(_lib, "load", lambda: fake)
    return fake


def _ints(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def _calls():
    """Every call that allocates: name, what it is given, and the call on a stream."""
    q = torch.zeros(2, 64, 512, dtype=torch.bfloat16, device="cuda")
    many = torch.zeros(300, 64, 512, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(64, ROW, dtype=torch.uint8, device="cuda")
    o_part = torch.zeros(2, 64, 3, 448, device="cuda")
    return {
        "decode": ([q, kv], lambda s, i: m.sparse_mla_decode(q, kv, i, num_splits=9, stream=s), _ints(2, 600)),
        "split": ([q, kv], lambda s, i: m.sparse_mla_decode_split(q, kv, i, 2, stream=s), _ints(2, 600)),
        "combine": ([o_part], lambda s, i: m.sparse_mla_combine(o_part, i, stream=s),
                    torch.zeros(2, 64, 3, device="cuda")),
        "noalloc": ([q, kv], lambda s, i: m.sparse_mla_decode_noalloc(q, kv, i, stream=s), _ints(2, 600)),
        "simt": ([q, kv], lambda s, i: m.sparse_mla_decode_simt(q, kv, i, stream=s), _ints(2, 600)),
        "paged": ([q, kv], lambda s, i: m.sparse_mla_decode_paged(q, kv, _ints(2, 4), 16, i, num_splits=9, stream=s),
                  _ints(2, 600)),
        "append": ([kv], lambda s, i: m.smla_cache_append(q[:, 0].contiguous(), kv, i, 16, _ints(3), _ints(2), stream=s),
                   _ints(2, 600)),
        "reserve": ([], lambda s, i: m.smla_cache_reserve(16, _ints(4), i, _ints(2), stream=s), _ints(2, 600)),
        "fork": ([kv], lambda s, i: m.smla_cache_fork(kv, 16, _ints(4), i, _ints(2), _ints(1), _ints(1), stream=s),
                 _ints(2, 600)),
        "free": ([], lambda s, i: m.smla_cache_free(_ints(4), _ints(2, 4), _ints(2), i, stream=s), _ints(900)),
        "compact": ([kv], lambda s, i: m.smla_cache_compact(kv, 16, _ints(4), i, stream=s), _ints(2, 600)),
        "chunk": ([q, kv], lambda s, i: m.smla_chunk_attention(q, kv, i, 16, _ints(3), _ints(2), max_kv_tokens=64, stream=s),
                  _ints(2, 600)),
        "chunk of many": ([many, kv], lambda s, i: m.smla_chunk_attention(many, kv, i, 16, _ints(3), _ints(2),
                                                                          max_kv_tokens=64, stream=s), _ints(2, 600)),
    }


NAMES = ["decode", "split", "combine", "noalloc", "simt", "paged", "append", "reserve", "fork", "free", "compact",
         "chunk", "chunk of many"]


def _owner(address):
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= address < seg["address"] + seg["total_size"]:
            return seg["stream"]
    return None


@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_allocates_belongs_to_its_stream(quiet, name):
    given, call, ints = _calls()[name]
    s = torch.cuda.Stream()
    ours = {t.data_ptr() for t in given + [ints]}
    result = call(s, ints)
    results = [t for t in (result if isinstance(result, tuple) else [result]) if t is not None]
    for t in results:
        assert _owner(t.data_ptr()) == s.cuda_stream
    if name not in ("append", "free", "split", "combine", "noalloc", "simt"):       # these take no workspace
        new = [a for a in quiet.seen if a not in ours and _owner(a) == s.cuda_stream]
        assert len(new) > len(results), "the workspace is not the stream's own"
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_an_argument_dropped_after_the_call_is_not_handed_out_again_early(quiet, name):
    _, call, ints = _calls()[name]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)              # about a tenth of a second
    call(s, ints)
    at, shape, dtype = ints.data_ptr(), ints.shape, ints.dtype
    del ints
    again = [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(256)]
    assert not s.query(), "the stream came to its end too soon for this test"
    assert at not in [t.data_ptr() for t in again]
    torch.cuda.synchronize()


@pytest.mark.parametrize("ns", [[1, 3], [150, 60]])
def test_attention_on_a_busy_stream_while_the_current_one_allocates(ns):
    """The call waits behind other work of its stream; memory that the current stream gets and
    fills meanwhile is not the call's."""
    page, H = 64, 64
    lens = [900, 500]
    num_pages = sum(-(-L // page) for L in lens) + 2
    pool, table = random_pool(num_pages, page, 5), tables(lens, page, num_pages, 5)
    cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    q = torch.randn(int(cu[-1]), H, 512, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    ref = chunk_reference(q, pool, table, page, cu, np.array(lens, np.int32))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    got = m.smla_chunk_attention(q, pool, dev(table), page, dev(cu), dev(np.array(lens, np.int32)), softmax_scale=SCALE,
                                 max_kv_tokens=sum(lens), stream=s)
    junk = [torch.full((1 << k,), -1, dtype=torch.int32, device="cuda") for k in (1, 2, 3, 7, 10, 16, 20, 22) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(s)
    check_chunk(got, ref)
    del junk


def test_page_calls_on_a_busy_stream_while_the_current_one_allocates():
    page, num_pages = 8, 64
    rng = np.random.default_rng(3)
    table = np.full((5, 4), -1, np.int32)
    order, at = rng.permutation(num_pages), 0
    lens = [30, 17, 8, 0, 0]
    ref = np.zeros(num_pages, np.int32)
    for r, L in enumerate(lens):
        k = -(-L // page)
        table[r, :k] = order[at:at + k]
        ref[order[at:at + k]] = 1
        at += k
    model = PageModel(ref, table, lens, page)
    r, t, l = dev(ref), dev(table), dev(np.array(lens, np.int32))
    pool = random_pool(num_pages, page, 12)
    want = pool.cpu().numpy().copy()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    m.smla_cache_free(r, t, l, dev(np.array([2], np.int32)), stream=s)
    m.smla_cache_fork(pool, page, r, t, l, dev(np.array([0, 0], np.int32)), dev(np.array([3, 4], np.int32)), stream=s)
    m.smla_cache_reserve(page, r, t, dev(np.array([32, 17, 9, 32, 31], np.int32)), stream=s)
    info = m.smla_cache_compact(pool, page, r, t, stream=s)
    junk = [torch.full((1 << k,), -1, dtype=torch.int32, device="cuda") for k in range(1, 12) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(s)
    model.free([2])
    model.fork([0, 0], [3, 4])
    model.reserve([32, 17, 9, 32, 31])
    assert info.cpu().tolist() == list(model.compact())
    check_pages(model, r, t, l)
    for a, b, rows in model.copies:
        want[b * page:b * page + rows] = want[a * page:a * page + rows]
    assert np.array_equal(pool.cpu().numpy(), want)
    del junk


def test_decode_on_a_busy_stream_while_the_current_one_allocates():
    w = W.Workload("side", 3, 64, 700, 4096, "uniform", seed=77)
    kv, q = W.make_cache(w, W.seq_lengths(w), device="cuda"), W.make_q(w, device="cuda")
    idx = torch.as_tensor(W.make_indices(w, W.seq_lengths(w)), device="cuda")
    want = m.sparse_mla_decode(q, kv, idx, num_splits=3)
    mine = idx.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    got = m.sparse_mla_decode(q, kv, mine, num_splits=3, stream=s)
    del mine
    junk = [torch.full((1 << k,), -1, dtype=torch.int32, device="cuda") for k in range(8, 22) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del junk


@pytest.mark.parametrize("ns", [[1, 3], [150, 60]])
def test_calls_on_a_stream_that_a_capture_forks_into(ns):
    """In a captured graph a call may run on a stream that was forked from the capture's, and
    allocate there; the graph's replays, and calls beside them, are right."""
    page, H = 64, 64
    lens = [900, 500]
    num_pages = sum(-(-L // page) for L in lens) + 2
    pool, table = random_pool(num_pages, page, 5), tables(lens, page, num_pages, 5)
    cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    q = torch.randn(int(cu[-1]), H, 512, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    args = (q, pool, dev(table), page, dev(cu), dev(np.array(lens, np.int32)))
    want = m.smla_chunk_attention(*args, softmax_scale=SCALE, max_kv_tokens=sum(lens))
    check_chunk(want, chunk_reference(q, pool, table, page, cu, np.array(lens, np.int32)))
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.wait_stream(torch.cuda.current_stream())
        here = m.smla_chunk_attention(*args, softmax_scale=SCALE, max_kv_tokens=sum(lens))
        there = m.smla_chunk_attention(*args, softmax_scale=SCALE, max_kv_tokens=sum(lens), stream=s)
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        for t in here + there:
            t.fill_(float("nan"))
        g.replay()
        beside = m.smla_chunk_attention(*args, softmax_scale=SCALE, max_kv_tokens=sum(lens))
        torch.cuda.synchronize()
        for got in (here, there, beside):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
