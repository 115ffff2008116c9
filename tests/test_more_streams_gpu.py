"""The append with a rotation, reading back, reordering, selection and the calls over 4-bit rows on
another stream than the current one, in captured graphs beside eager calls, and after a wait has run
out."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_mla_decode_03_gb300 as m
from sparse_mla_decode_03_gb300 import _lib

from _cache_helpers import PageModel, SCALE, check_chunk, check_pages, dev, tables
from _rows4_helpers import (ROW4, chunk_reference4, dequantize4, random_pool4, reorder_model, rotary_table, rotate64,
                            select_reference)

pytestmark = pytest.mark.gpu


class NoLaunch:
    """The library with entry points that note the addresses they get and do nothing."""

    def __init__(self, lib):
        self.lib, self.seen = lib, []

    def __getattr__(self, name):
        if name.endswith("_size") or name in ("smla_default_num_splits", "smla_status_string"):
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
    """Name: what the call is given, the call on a stream with an argument of its own, that argument, and whether
    it takes a workspace."""
    q = torch.zeros(2, 64, 512, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(64, ROW4, dtype=torch.uint8, device="cuda")
    rows = torch.zeros(2, 512, dtype=torch.bfloat16, device="cuda")
    turn = torch.zeros(40, 64, device="cuda")
    logits = torch.zeros(6, 2000, device="cuda")
    return {
        "decode": ([q, kv], lambda s, i: m.sparse_mla_decode(q, kv, i, stream=s), _ints(2, 600), True),
        "paged": ([q, kv], lambda s, i: m.sparse_mla_decode_paged(q, kv, _ints(2, 4), 16, i, stream=s), _ints(2, 600), True),
        "chunk": ([q, kv], lambda s, i: m.smla_chunk_attention(q, kv, i, 16, _ints(3), _ints(2), max_kv_tokens=64, stream=s),
                  _ints(2, 600), True),
        "rotary": ([rows, kv, turn], lambda s, i: m.smla_cache_append_rotary(rows, kv, i, 16, _ints(3), _ints(2), turn, stream=s),
                   _ints(2, 600), False),
        "read": ([kv], lambda s, i: m.smla_cache_read(kv, i, 16, _ints(3), _ints(2), 9, stream=s), _ints(2, 600), False),
        "reorder": ([kv], lambda s, i: m.smla_cache_reorder(kv, 16, _ints(4), i, _ints(2), _ints(2), stream=s), _ints(2, 600), True),
        "select": ([logits], lambda s, i: m.smla_beam_select(logits, i.view(torch.float32), stream=s), _ints(2, 3), True),
    }


NAMES = ["decode", "paged", "chunk", "rotary", "read", "reorder", "select"]


def _owner(address):
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= address < seg["address"] + seg["total_size"]:
            return seg["stream"]
    return None


@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_allocates_belongs_to_its_stream(quiet, name):
    given, call, ints, workspace = _calls()[name]
    s = torch.cuda.Stream()
    ours = {t.data_ptr() for t in given + [ints]}
    result = call(s, ints)
    results = [t for t in (result if isinstance(result, tuple) else [result]) if t is not None]
    for t in results:
        assert _owner(t.data_ptr()) == s.cuda_stream
    if workspace:
        new = [a for a in quiet.seen if a not in ours and _owner(a) == s.cuda_stream]
        assert len(new) > len(results), "the workspace is not the stream's own"
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_an_argument_dropped_after_the_call_is_not_handed_out_again_early(quiet, name):
    _, call, ints, _ = _calls()[name]
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


def test_a_step_on_a_busy_stream_and_in_a_graph_beside_it():
    """Append, attention, selection and reordering on a stream that other work holds up, while the current one
    allocates; then captured, with calls of the same kind beside the replays."""
    page, H, lens = 16, 64, [70, 33]
    num_pages = 20
    table = tables(lens, page, num_pages, 3)
    ref = np.zeros(num_pages, np.int32)
    ref[table[table >= 0]] = 1
    start = random_pool4(num_pages, page, 4)
    turn = rotary_table(100)
    kv = torch.randn(2, 512, device="cuda").to(torch.bfloat16)
    q_rope, q = torch.randn(2, H, 64, device="cuda").to(torch.bfloat16), torch.randn(2, H, 512, device="cuda").to(torch.bfloat16)
    logits, scores = torch.randn(2, 5000, device="cuda") * 2, torch.tensor([[-1.0, -1.5]], device="cuda")
    cu = dev(np.array([0, 1, 2], np.int32))
    pool, r, t, l = start.clone(), dev(ref), dev(table), dev(np.array(lens, np.int32))

    def step(s=None):
        m.smla_cache_append_rotary(kv, pool, t, page, cu, l, turn, q_rope=q_rope, q=q, stream=s)
        back = m.smla_cache_read(pool, t, page, cu, l, 2, stream=s)
        out = m.smla_chunk_attention(q, pool, t, page, cu, l, softmax_scale=SCALE, stream=s)
        best = m.smla_beam_select(logits, scores, stream=s)
        m.smla_cache_reorder(pool, page, r, t, l, best[0].view(-1), stream=s)
        return back, out, best

    def check(got):
        (back, out, (parents, tokens, values)), model = got, PageModel(ref, table, lens, page)
        p, k, v = select_reference(logits, scores, 2)
        assert np.array_equal(parents.cpu().numpy(), p) and np.array_equal(tokens.cpu().numpy(), k)
        reorder_model(model, p.reshape(-1).tolist())
        check_pages(model, r, t, l)
        # the pool as the append left it, before the copies
        rows = start.clone()
        at = [table[b, (L - 1) // page] * page + (L - 1) % page for b, L in enumerate(lens)]
        kept = [pool[i] if not any(a * page <= i < a * page + n for _, a, n in model.copies) else None for i in at]
        for i, row in zip(at, kept):
            rows[i] = row
        nope, rope = dequantize4(rows[at].cpu().numpy())
        assert np.array_equal(back.double().cpu().numpy(), np.concatenate([nope, rope], axis=1))
        want, tol = rotate64(kv[:, 448:], turn[[L - 1 for L in lens]], True)
        assert ((back[:, 448:].double() - want).abs() <= tol).all()
        check_chunk(out, chunk_reference4(q, rows, table, page, np.array([0, 1, 2]), np.array(lens)))

    def reset():
        pool.copy_(start)
        r.copy_(dev(ref))
        t.copy_(dev(table))
        l.copy_(dev(np.array(lens, np.int32)))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    got = step(s)
    junk = [torch.full((1 << k,), -1, dtype=torch.int32, device="cuda") for k in range(1, 22) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(s)
    check(got)
    reset()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    beside = torch.randn(6, 30000, device="cuda")
    for _ in range(3):
        reset()
        g.replay()
        others = m.smla_beam_select(beside, torch.zeros(2, 3, device="cuda"), 6)
        torch.cuda.synchronize()
        check(got)
        want = select_reference(beside, torch.zeros(2, 3), 6)
        assert np.array_equal(others[1].cpu().numpy(), want[1])
    del junk


@pytest.mark.parametrize("block", [0, 1])
@pytest.mark.parametrize("n", [1, 40])
def test_a_wait_that_runs_out(block, n):
    """One warp withholds its signal: the call returns, the status says so, and the next call is right."""
    page, H, lens = 64, 64, [3000, 20000]
    num_pages = sum(-(-L // page) for L in lens) + 2
    pool, table = random_pool4(num_pages, page, 7), tables(lens, page, num_pages, 7)
    cu = np.array([0, n, 2 * n], np.int32)
    q = torch.randn(2 * n, H, 512, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    args = (q, pool, dev(table), page, dev(cu), dev(np.array(lens, np.int32)))
    lib = m._lib.load()
    m.smla_device_status(clear=True)
    assert lib.smla_test_inject_fault(block) == 0
    try:
        m.smla_chunk_attention(*args)
        torch.cuda.synchronize()
        assert m.smla_device_status(clear=True) == m._lib.SMLA_ERR_TIMEOUT
        if n == 1:
            m.sparse_mla_decode(q, pool, dev(np.arange(2 * 2000, dtype=np.int32).reshape(2, -1)))
            torch.cuda.synchronize()
            assert m.smla_device_status(clear=True) == m._lib.SMLA_ERR_TIMEOUT
    finally:
        assert lib.smla_test_inject_fault(-1) == 0
    got = m.smla_chunk_attention(*args, softmax_scale=SCALE)
    assert m.smla_device_status(clear=True) == 0
    check_chunk(got, chunk_reference4(q, pool, table, page, cu, np.array(lens, np.int32)))


def test_refusals_of_tensors_on_the_gpu():
    kv = torch.zeros(4, 512, dtype=torch.bfloat16, device="cuda")
    pool, turn = torch.zeros(64, ROW4, dtype=torch.uint8, device="cuda"), torch.zeros(8, 64, device="cuda")
    t, cu, l = _ints(2, 4), _ints(3), _ints(2)
    q, r = torch.zeros(4, 3, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 3, 64, dtype=torch.bfloat16, device="cuda")

    def rotary(kv=kv, pool=pool, turn=turn, q=q, r=r, **kw):
        m.smla_cache_append_rotary(kv, pool, t, 16, cu, l, turn, q_rope=r, q=q, **kw)

    logits, scores = torch.zeros(6, 50, device="cuda"), torch.zeros(2, 3, device="cuda")
    wrong = [lambda: rotary(q=None), lambda: rotary(r=None), lambda: rotary(q=q[:3]), lambda: rotary(q=q[:, :2]),
             lambda: rotary(q=q.float()), lambda: rotary(r=r[:, :, ::2]), lambda: rotary(turn=turn[:, :63]),
             lambda: rotary(turn=turn.double()), lambda: rotary(q=q[:, :1].expand(4, 3, 512)),
             lambda: rotary(q=q[:1].expand(4, 3, 512)),
             lambda: rotary(q=torch.zeros(4000, dtype=torch.bfloat16, device="cuda").as_strided((4, 3, 512), (512, 512, 1))),
             lambda: rotary(pool=pool[:, :360]), lambda: rotary(kv=kv[:, :511]), lambda: rotary(turn=turn.cpu()),
             lambda: m.smla_cache_read(pool, t, 16, cu, l, 5, out=kv),
             lambda: m.smla_cache_read(pool, t, 16, cu, l, 4, out=kv.float()),
             lambda: m.smla_cache_reorder(pool, 16, _ints(4), t, l, _ints(3)),
             lambda: m.smla_cache_reorder(pool, 16, _ints(5), t, l, _ints(2)),
             lambda: m.smla_cache_reorder(pool, 16, _ints(4), t, l, _ints(2).long()),
             lambda: m.smla_beam_select(logits[:5], scores), lambda: m.smla_beam_select(logits.t(), scores),
             lambda: m.smla_beam_select(logits, scores.double()), lambda: m.smla_beam_select(logits, scores.t()),
             lambda: m.smla_beam_select(logits, scores, finished=_ints(6)),
             lambda: m.smla_beam_select(logits, scores, finished=torch.zeros(5, dtype=torch.bool, device="cuda")),
             lambda: m.smla_beam_select(logits, scores, 4, parents=_ints(2, 3)),
             lambda: m.smla_beam_select(logits, scores, out_scores=_ints(2, 3))]
    refused = [lambda: m.smla_beam_select(logits, scores, 65), lambda: m.smla_beam_select(logits, scores, 0),
             lambda: m.smla_beam_select(logits, scores, finished=torch.zeros(6, dtype=torch.bool, device="cuda"), end_token=50),
             lambda: m.smla_beam_select(logits[:1].expand(6, 50), scores),          # rows on one another
             lambda: rotary(turn=torch.zeros(8 * 64 + 2, device="cuda")[2:].view(8, 64)),
             lambda: m.sparse_mla_decode(q[:2].new_zeros(2, 16, 512), pool, _ints(2, 64), num_splits=2)]
    for calls, error in ((wrong, ValueError), (refused, m.SmlaError)):
        for i, call in enumerate(calls):
            try:
                call()
            except error:
                continue
            pytest.fail(f"{error.__name__}: call {i} was taken")


def test_calls_on_two_streams_at_once():
    """Each call has a workspace of its own, so that calls in flight together do not meet."""
    page, lens = 64, [5000, 12000, 700]
    num_pages = sum(-(-L // page) for L in lens) + 4
    pool, table = random_pool4(num_pages, page, 8), dev(tables(lens, page, num_pages, 8))
    l, cu1, cu40 = dev(np.array(lens, np.int32)), dev(np.arange(4).astype(np.int32)), dev(40 * np.arange(4).astype(np.int32))
    g = torch.Generator(device="cuda").manual_seed(8)
    q1, q40 = (torch.randn(n, 64, 512, generator=g, device="cuda").to(torch.bfloat16) for n in (3, 120))
    idx = torch.randint(-1, pool.shape[0], (20, 1500), generator=g, device="cuda", dtype=torch.int32)
    qs = torch.randn(20, 64, 512, generator=g, device="cuda").to(torch.bfloat16)
    logits, scores = torch.randn(48, 60001, generator=g, device="cuda"), torch.randn(6, 8, generator=g, device="cuda")
    jobs = [lambda: m.smla_chunk_attention(q1, pool, table, page, cu1, l, softmax_scale=SCALE, max_kv_tokens=sum(lens)),
            lambda: m.smla_chunk_attention(q40, pool, table, page, cu40, l, softmax_scale=SCALE, max_kv_tokens=sum(lens)),
            lambda: m.sparse_mla_decode(qs, pool, idx), lambda: m.smla_beam_select(logits, scores),
            lambda: (m.smla_cache_read(pool, table, page, cu40, l, 120),)]
    want = [[t.clone() for t in job()] for job in jobs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for turn in range(6):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append([(i, jobs[i]()) for i in (range(len(jobs)) if k == 0 else reversed(range(len(jobs))))])
    torch.cuda.synchronize()
    for results in got:
        for i, r in results:
            for a, b in zip(r, want[i]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
