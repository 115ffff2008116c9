"""smla_beam_select against the definition in 64 bits: parents and tokens exactly, values within the
bound derived in _rows4_helpers; and a beam-searched run of the calls that belong together."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_03_gb300 as m

from _cache_helpers import PageModel, ROW, SCALE, check_chunk, chunk_reference, dev
from _rows4_helpers import ROW4, chunk_reference4, reorder_model, rotary_table, select_reference

pytestmark = pytest.mark.gpu
INF = float("inf")


def _logits(G, K, V, seed, dtype=torch.float32, pad=0, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(G * K, V + pad, generator=g, device="cuda") * spread
    scores = -20.0 * torch.rand(G, K, generator=g, device="cuda")
    return x.to(dtype)[:, pad // 2:pad // 2 + V], scores


def _check(logits, scores, n=None, finished=None, end=0, status=0, **kw):
    m.smla_device_status(clear=True)
    got = m.smla_beam_select(logits, scores, num_out=n, finished=finished, end_token=end, **kw)
    assert m.smla_device_status(clear=True) == status
    want = select_reference(logits, scores, n or scores.shape[1], finished, end)
    _same(got, want)
    return got


def _same(got, want):
    parents, tokens, values = (t.cpu().numpy() for t in got)
    assert np.array_equal(parents, want[0])
    assert np.array_equal(tokens, want[1])
    none = want[0] < 0
    assert np.isneginf(values[none]).all()
    d = np.abs(values[~none].astype(np.float64) - want[2][~none])
    tol = 2.0 ** -16 + 2.0 ** -24 * np.abs(want[2][~none])
    assert (d <= tol).all(), f"worst error / tolerance {(d / tol).max():.3g}"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("G,K,n,V,pad", [
    (1, 1, 1, 1, 0), (1, 1, 1, 2, 1), (3, 2, 2, 5, 0), (2, 4, 8, 31, 3), (5, 3, 3, 257, 1), (1, 4, 4, 32000, 0),
    (7, 5, 10, 8191, 1), (2, 8, 16, 8192, 0), (2, 8, 16, 8193, 7), (2, 12, 24, 50257, 2), (1, 64, 64, 16400, 5),
    (3, 33, 40, 1000, 0), (2, 1, 64, 20000, 0), (4, 6, 9, 131071, 0),
])
def test_random(dtype, G, K, n, V, pad):
    logits, scores = _logits(G, K, V, V + n, dtype, pad)
    _check(logits, scores, n)


def test_rows_that_begin_anywhere():
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        flat = torch.randn(6 * 9001 + 16, device="cuda").to(dtype)
        for at in range(9):
            logits = flat[at:at + 6 * 9001].view(6, 9001)
            _check(logits, torch.zeros(2, 3, device="cuda") - torch.arange(3, device="cuda"), 5)


@pytest.mark.parametrize("V", [3, 40, 9000])
def test_fewer_candidates_than_wanted(V):
    logits, scores = _logits(2, 2, V, 3)
    logits[:, 2:] = -INF
    _check(logits, scores, 16)
    logits[1] = -INF
    _check(logits, scores, 16)
    logits[:] = -INF
    _check(logits, scores, 4)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_masks_of_the_type_s_lowest_value(dtype):
    logits, scores = _logits(2, 3, 20000, 4, dtype)
    low = torch.finfo(dtype).min
    logits[:, ::3] = low
    _check(logits, scores, 6)
    logits[0] = low                                       # uniform, far down
    logits[4, 10:] = low
    _check(logits, scores, 12)


@pytest.mark.parametrize("n", [1, 8, 40, 64])
def test_equal_logits(n):
    """The lowest token first, however many are equal; all equal, in part, in steps."""
    scores = torch.tensor([[-1.0, -2.0]], device="cuda")
    for V in (70, 8192, 20001):
        x = torch.zeros(2, V, device="cuda")
        _check(x, scores, n)
        _check(x.bfloat16() + 7.5, scores, n)
        x[:, V // 2:] = 1.0
        _check(x, scores, n)
        x[:] = -(torch.arange(V, device="cuda") // 50).float()
        _check(x, scores, n)
        x[0, ::2] = -0.0
        x[0, 1::2] = 0.0
        _check(x, scores, n)


@pytest.mark.parametrize("n", [4, 16, 64])
def test_sorted_logits(n):
    """All of the largest in one thread's or one part's hands."""
    for V in (8192, 30000):
        up = torch.linspace(-9, 9, V, device="cuda").expand(2, V).contiguous()
        scores = torch.tensor([[-3.0, -3.5]], device="cuda")
        _check(up, scores, n)
        _check(up.flip(1).contiguous(), scores, n)
        x = torch.full((2, V), -50.0, device="cuda")
        for first in range(0, 400, 8):
            x[0, first * 8 % V] = first / 10.0
        x[1, 256:512] = torch.arange(256, device="cuda") / 16
        _check(x, scores, n)


def test_beams_that_tie():
    logits, _ = _logits(1, 1, 5000, 6)
    logits = logits.expand(4, 5000).contiguous()
    _check(logits, torch.full((1, 4), -2.5, device="cuda"), 10)
    _check(logits, torch.tensor([[-2.5, -INF, -2.5, -2.5]], device="cuda"), 3)


def test_scores_and_logits_that_are_not_finite():
    logits, scores = _logits(3, 3, 9000, 7)
    scores[0, 1] = -INF                                   # a beam that is not there yet: no error
    scores[1] = -INF
    _check(logits, scores, 5)
    for what in (INF, float("nan")):
        x = logits.clone()
        x[7, 8500] = what
        _check(x, scores, 5, status=-8)
        x = torch.full_like(logits, -INF)
        x[4:, 77] = 1.0
        x[8, 8999] = what
        _check(x, torch.zeros(3, 3, device="cuda"), 5, status=-8)
        s = scores.clone()
        s[2, 2] = what
        _check(logits, s, 5, status=-8)
    x = logits.clone()
    x[5] = float("nan")
    _check(x, torch.zeros(3, 3, device="cuda"), 5, status=-8)


def test_logits_of_any_size():
    logits, scores = _logits(2, 2, 6000, 8)
    for scale in (1e-4, 1e3, 1e30, 1e37):
        _check(logits * scale, scores, 4)
    _check(logits + 1e6, scores, 4)


@pytest.mark.parametrize("kind", [torch.uint8, torch.bool])
def test_finished_beams(kind):
    logits, scores = _logits(4, 5, 700, 9)
    done = torch.zeros(20, device="cuda")
    done[[1, 3, 10, 11, 12, 13, 14]] = 1
    logits[3] = float("nan")                              # not read
    scores[0, 1] = 1.0
    scores[2, 2] = -INF
    _check(logits, scores, 7, done.to(kind), 699)
    s = scores.clone()
    s[0, 1] = INF
    _check(logits, s, 7, done.to(kind), 699, status=-8)


def test_replay_and_repetition():
    logits, scores = _logits(3, 4, 40000, 10, torch.bfloat16)
    p = m.make_beam_params(3, 4, 40000, 8, logits_type=1)
    ws = torch.empty(m.smla_beam_workspace_size(p), dtype=torch.uint8, device="cuda")
    a = m.smla_beam_select(logits, scores, 8, workspace=ws)
    b = m.smla_beam_select(logits, scores, 8)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        m.smla_beam_select(logits, scores, 8, parents=a[0], tokens=a[1], out_scores=a[2], workspace=ws)
    for seed in (11, 12):
        x, c = _logits(3, 4, 40000, seed, torch.bfloat16)
        logits.copy_(x)
        scores.copy_(c)
        g.replay()
        torch.cuda.synchronize()
        _same(a, select_reference(logits, scores, 8))


def test_rows_past_32_bits_of_offset():
    V, R = 1 << 20, 2100
    if torch.cuda.mem_get_info()[0] < 3 * V * R * 2:
        pytest.skip("not enough memory")
    logits = torch.zeros(R, V, dtype=torch.bfloat16, device="cuda")
    logits[:, 5] = 1.0
    logits[2099, 1000000] = 9.0
    scores = torch.zeros(R // 2, 2, device="cuda")
    parents, tokens, values = m.smla_beam_select(logits, scores, 1)
    assert tokens[:-1].eq(5).all() and tokens[-1].item() == 1000000
    assert parents.view(-1)[:-1].tolist() == list(range(0, R - 2, 2)) and parents[-1].item() == R - 1


@pytest.mark.parametrize("row", [ROW, ROW4])
def test_a_beam_searched_run(row):
    """Prompts, then steps of: room for a token, its row and queries rotated into place, attention,
    selection, reordering.  Each step's results are checked against the definitions over the tokens
    that each beam really has, which a list beside the cache follows."""
    G, K, H, page, V, max_pages = 2, 3, 16, 8, 300, 6
    R = G * K
    g = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    num_pages = R * max_pages
    pool = torch.zeros(num_pages * page, row, dtype=torch.uint8, device="cuda")
    ref = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
    table = torch.full((R, max_pages), -1, dtype=torch.int32, device="cuda")
    embed = normal(V, 512).to(torch.bfloat16)             # a token's row before the rotation
    ask = normal(V, H, 512).to(torch.bfloat16)
    head = normal(H * 448, V) * 0.02
    turn = rotary_table(64)
    prompts = [[int(t) for t in torch.randint(0, V, (n,), generator=g, device="cuda")] for n in (13, 9)]
    # the prompt of a group in its first row; the reordering makes the others
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    lens[::K] = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
    m.smla_device_status(clear=True)
    m.smla_cache_reserve(page, ref, table, lens)
    tokens = torch.tensor([t for p in prompts for t in p], device="cuda")
    cu = np.concatenate([[0], np.cumsum([len(prompts[r // K]) if r % K == 0 else 0 for r in range(R)])]).astype(np.int32)
    m.smla_cache_append_rotary(embed[tokens], pool, table, page, dev(cu), lens, turn)
    m.smla_cache_reorder(pool, page, ref, table, lens, dev(np.array([r // K * K for r in range(R)], np.int32)))
    paths = [list(prompts[r // K]) for r in range(R)]
    scores = torch.tensor([[0.0] + [-INF] * (K - 1)] * G, device="cuda")
    last = torch.tensor([p[-1] for p in paths], device="cuda")
    step_cu = dev(np.arange(R + 1).astype(np.int32))
    reference = chunk_reference if row == ROW else chunk_reference4
    for step in range(9):
        lens += 1
        m.smla_cache_reserve(page, ref, table, lens)
        q = ask[last].clone()
        m.smla_cache_append_rotary(embed[last], pool, table, page, step_cu, lens, turn, q_rope=ask[last][:, :, 448:], q=q)
        for r in range(R):
            paths[r].append(int(last[r]))
        out, lse = m.smla_chunk_attention(q, pool, table, page, step_cu, lens, softmax_scale=SCALE)
        # the same tokens in a cache of their own, appended in one call
        count = R * max_pages
        fresh = torch.zeros(count * page, row, dtype=torch.uint8, device="cuda")
        own = np.arange(count).reshape(R, max_pages).astype(np.int32)
        own_cu = np.concatenate([[0], np.cumsum([len(p) for p in paths])]).astype(np.int32)
        m.smla_cache_append_rotary(embed[torch.tensor([t for p in paths for t in p], device="cuda")], fresh, dev(own), page,
                                   dev(own_cu), lens, turn)
        check_chunk((out, lse), reference(q, fresh, own, page, np.arange(R + 1), lens.cpu().numpy()))
        logits = out.float().reshape(R, -1) @ head
        parents, chosen, new = m.smla_beam_select(logits, scores)
        _same((parents, chosen, new), select_reference(logits, scores, K))
        scores = new
        m.smla_cache_reorder(pool, page, ref, table, lens, parents.view(-1))
        paths = [list(paths[p]) for p in parents.view(-1).tolist()]
        last = chosen.view(-1).long()
    assert m.smla_device_status(clear=True) == 0
    # every page is counted as often as it is listed
    counts = torch.bincount(table[table >= 0].long(), minlength=num_pages)
    assert torch.equal(counts.int(), ref)


def test_scores_that_are_replaced_where_they_lie():
    logits, scores = _logits(40, 8, 5000, 5)
    want = select_reference(logits, scores, 8)
    got = m.smla_beam_select(logits, scores, out_scores=scores)
    assert got[2] is scores
    _same(got, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G,K,n,V", [(5, 8, 16, 11306), (4, 9, 18, 1054), (3, 7, 7, 1850), (2, 10, 10, 112), (2, 64, 64, 600), (1, 3, 6, 224)])
def test_few_steps_and_beams_far_apart(G, K, n, V, dtype):
    """The best come from one or two beams, whose steps are fewer than the results."""
    logits, scores = _logits(G, K, V, V, dtype)
    _check(logits, scores * 4, n)
    done = torch.zeros(G * K, dtype=torch.uint8, device="cuda")
    done[::3] = 1
    _check(logits, scores * 4, n, done, 2)


def test_more_equal_steps_than_are_read_again():
    logits = torch.full((24, 60000), -1.5, device="cuda")
    logits[5, 59999] = 3.0
    logits[17, 1024] = 2.0
    scores = torch.zeros(2, 12, device="cuda")
    scores[1] -= torch.arange(12, device="cuda") * 0.5
    _check(logits, scores, 24)
    lowest = torch.finfo(torch.bfloat16).min
    logits = torch.full((16, 70000), lowest, dtype=torch.bfloat16, device="cuda")
    logits[:, 69000:69003] = 1.0
    _check(logits, torch.zeros(2, 8, device="cuda"), 40)
