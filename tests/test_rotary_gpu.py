"""smla_cache_append_rotary against the rotation in 64 bits (tolerance: _rows4_helpers) and, for the
bytes that no rotation touches, against smla_cache_append's definition."""
import numpy as np
import pytest
import torch

import sparse_mla_decode_03_gb300 as m

from _cache_helpers import ROW, dev, pack_rows, random_pool, tables
from _rows4_helpers import ROW4, pack_rows4, random_pool4, rotary_table, rotate64

pytestmark = pytest.mark.gpu


def _ints(v):
    return dev(np.asarray(v, np.int32))


def _rope_of(rows):
    at = 456 if rows.shape[1] >= ROW else 240
    return torch.as_tensor(np.ascontiguousarray(rows[:, at:at + 128])).view(torch.bfloat16).cuda()


def _near(got, want, tol):
    d = (got.double() - want).abs()
    assert (d <= tol).all(), f"worst error / tolerance {(d / tol).max().item():.3g}"


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("lens,ns,page,H", [
    ([1], [1], 1, 1),
    ([5, 40, 17], [5, 1, 17], 16, 5),
    ([100, 33, 64, 7], [64, 0, 1, 7], 48, 16),
    ([130] * 20, [3] * 20, 64, 17),
    ([4000, 900], [70, 2], 64, 64),
    ([300], [130], 64, 0),
])
def test_rows_and_queries(interleaved, bits, lens, ns, page, H):
    num_pages = sum(-(-L // page) for L in lens) + 3
    pool = (random_pool if bits == 8 else random_pool4)(num_pages, page, 7)
    table = tables(lens, page, num_pages, 7)
    T = sum(ns)
    cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    g = torch.Generator().manual_seed(T + H)
    kv = torch.randn(T, 520, generator=g).to(torch.bfloat16).cuda()[:, :512]
    turn = rotary_table(max(lens))
    wide = torch.randn(T, max(H, 1), 72, generator=g).to(torch.bfloat16).cuda()
    q_rope = wide[:, :H, :64]
    q = torch.full((T, H, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    want = pool.cpu().numpy().copy()
    pos = np.concatenate([np.arange(L - n, L) for L, n in zip(lens, ns)])
    at = np.concatenate([[table[b, p // page] * page + p % page for p in range(L - n, L)]
                         for b, (L, n) in enumerate(zip(lens, ns))]).astype(np.int64)
    m.smla_device_status(clear=True)
    m.smla_cache_append_rotary(kv, pool, dev(table), page, dev(cu), _ints(lens), turn, interleaved=interleaved,
                               q_rope=q_rope if H else None, q=q if H else None)
    assert m.smla_device_status(clear=True) == 0
    got = pool.cpu().numpy()
    t = turn[torch.as_tensor(pos, device="cuda")]
    _near(_rope_of(got[at]), *rotate64(kv[:, 448:], t, interleaved))
    width, first = (ROW, 456) if bits == 8 else (ROW4, 240)
    want[at, :first] = (pack_rows if bits == 8 else pack_rows4)(kv)[:, :first]
    want[at, first:width] = got[at, first:width]
    assert np.array_equal(got, want)
    if H:
        _near(q[:, :, 448:], *rotate64(q_rope, t[:, None], interleaved))
        assert (q[:, :, :448] == 5).all()


def test_a_rotation_by_nothing_is_the_append():
    page, T = 16, 33
    kv = torch.randn(T, 512, device="cuda").to(torch.bfloat16)
    turn = torch.cat([torch.ones(T, 32), torch.zeros(T, 32)], dim=1).cuda()
    for row in (ROW, ROW4):
        a, b = (torch.zeros(64, row, dtype=torch.uint8, device="cuda") for _ in range(2))
        args = (_ints([[3, 1, 0]]), page, _ints([0, T]), _ints([T]))
        m.smla_cache_append(kv, a, *args)
        for pairs in (True, False):
            b.zero_()
            m.smla_cache_append_rotary(kv, b, *args, turn, interleaved=pairs)
            assert torch.equal(a, b)


def test_tokens_without_a_place_a_rotation_or_a_sequence():
    """Positions past the table of rotations or below 0: row and queries untouched, reported; no page:
    queries rotated, reported; outside every sequence: untouched, not reported."""
    page, T, H = 8, 14, 3
    pool = random_pool4(6, page, 3)
    before = pool.cpu().numpy().copy()
    turn = rotary_table(16)
    kv = torch.randn(T, 512, device="cuda").to(torch.bfloat16)
    q_rope = torch.randn(T, H, 64, device="cuda").to(torch.bfloat16)
    table = np.array([[0, -1, 2], [1, 3, 4], [5, -1, -1]], np.int32)
    cu, lens = [1, 5, 9, 12], [10, 18, 2]
    # sequence 0: positions 6..9 (8, 9 unmapped); 1: 14..17 (16, 17 without a rotation); 2: -1..1
    q = torch.full((T, H, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    m.smla_device_status(clear=True)
    m.smla_cache_append_rotary(kv, pool, dev(table), page, _ints(cu), _ints(lens), turn, q_rope=q_rope, q=q)
    assert m.smla_device_status(clear=True) == -7
    pos = {1: 6, 2: 7, 3: 8, 4: 9, 5: 14, 6: 15, 10: 0, 11: 1}
    rows = {1: 6, 2: 7, 5: 30, 6: 31, 10: 40, 11: 41}
    got = pool.cpu().numpy()
    touched = sorted(rows.values())
    rest = [r for r in range(48) if r not in touched]
    assert np.array_equal(got[rest], before[rest])
    for t in range(T):
        if t in rows:
            assert np.array_equal(got[rows[t], :240], pack_rows4(kv[t:t + 1])[0, :240])
            _near(_rope_of(got[rows[t]:rows[t] + 1]), *rotate64(kv[t:t + 1, 448:], turn[pos[t]][None], True))
        if t in pos:
            _near(q[t, :, 448:], *rotate64(q_rope[t], turn[pos[t]][None], True))
        else:
            assert (q[t] == 5).all()


def test_strided_queries_and_replay():
    """Queries head-major, q inside a wider buffer; a captured call follows new lengths."""
    T, H, page = 6, 20, 16
    pool = random_pool4(30, page, 1)
    table = tables([200, 200], page, 30, 1)
    turn = rotary_table(200)
    kv = torch.randn(T, 512, device="cuda").to(torch.bfloat16)
    q_rope = torch.randn(H, T, 64, device="cuda").to(torch.bfloat16).transpose(0, 1)
    store = torch.zeros(T, H, 528, dtype=torch.bfloat16, device="cuda")
    q, lens, t, cu = store[:, :, 8:520], _ints([50, 60]), dev(table), _ints([0, 3, T])

    def call():
        m.smla_cache_append_rotary(kv, pool, t, page, cu, lens, turn, interleaved=False, q_rope=q_rope, q=q)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for new in ([50, 60], [199, 3], [70, 200]):
        lens.copy_(_ints(new))
        store.zero_()
        g.replay()
        torch.cuda.synchronize()
        pos = torch.as_tensor(np.concatenate([np.arange(L - 3, L) for L in new]), device="cuda")
        _near(q[:, :, 448:], *rotate64(q_rope, turn[pos][:, None], False))
        assert (store[:, :, :456] == 0).all() and (store[:, :, 520:] == 0).all()


@pytest.mark.parametrize("interleaved", [True, False])
def test_queries_rotated_where_they_lie(interleaved):
    pool = random_pool4(8, 16, 3)
    turn = rotary_table(128)
    q = torch.randn(5, 33, 512, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    before = q.clone()
    lens = [40, 77]
    m.smla_cache_append_rotary(q.new_zeros(5, 512), pool, dev(tables(lens, 16, 8, 3)), 16, _ints([0, 2, 5]), _ints(lens), turn,
                               interleaved=interleaved, q_rope=q[:, :, 448:], q=q)
    at = torch.tensor([38, 39, 74, 75, 76], device="cuda")
    _near(q[:, :, 448:], *rotate64(before[:, :, 448:], turn[at][:, None], interleaved))
    assert torch.equal(q[:, :, :448], before[:, :, :448])
