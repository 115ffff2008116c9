"""smla_beam_select where many candidates are equal, and over wide groups, against the definition in 64
bits (tolerances: _rows4_helpers).  Where candidates are equal, sums are whole numbers and powers of two,
so that ties are exact."""
import math

import pytest
import torch

import sparse_mla_decode_03_gb300 as m

from test_beam_gpu import _check, _logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("live,each", [(32, 16), (33, 16), (17, 32), (9, 64), (37, 16)])
@pytest.mark.parametrize("ended", [0, 1, 3])
def test_a_few_more_equal_candidates_than_are_ranked(dtype, live, each, ended):
    """512 to 592 equal candidates of a group above all others, beside finished beams whose value is
    the same in 32 bits, and which have no logits to wait for."""
    G, K, V = 5, live + ended, 8000
    g = torch.Generator(device="cuda").manual_seed(live + each)
    logits = torch.full((G * K, V), torch.finfo(dtype).min, dtype=dtype, device="cuda")
    done = torch.zeros(G, K, dtype=torch.uint8, device="cuda")
    for group in range(G):
        done[group, torch.randperm(K, generator=g, device="cuda")[:ended]] = 1
    for row in (done.view(-1) == 0).nonzero().view(-1).tolist():
        logits[row, torch.randperm(V, generator=g, device="cuda")[:each]] = 2.0
    scores = torch.where(done == 1, -math.log(each), 0.0).float()
    for n in (1, 8, 64):
        _check(logits, scores, n, done.view(-1), V - 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_constant_rows_beside_finished_beams(dtype):
    G, K, V = 24, 6, 1 << 13
    logits = torch.full((G * K, V), 0.5, device="cuda").to(dtype)
    done = torch.zeros(G, K, dtype=torch.uint8, device="cuda")
    done[:, ::3] = 1
    scores = torch.where(done == 1, -math.log(V), 0.0).float()
    for n in (2, 24, 64):
        _check(logits, scores, n, done.view(-1), 7)


@pytest.mark.parametrize("G,K,n,V,dtype", [
    (2, 64, 64, 131072, torch.bfloat16), (2, 32, 64, 131072, torch.float32), (1, 64, 64, 131072, torch.float16),
    (2, 48, 33, 100001, torch.float32), (3, 16, 64, 262143, torch.float32),
])
def test_wide_groups_whose_beams_are_far_apart(G, K, n, V, dtype):
    """The best come from a few beams, nearly all of whose steps reach a border that few threads' maxima
    make."""
    logits, scores = _logits(G, K, V, V + K, dtype)
    _check(logits, scores * 4, n)
    done = torch.zeros(G, K, dtype=torch.uint8, device="cuda")
    done[:, 5::9] = 1
    _check(logits, scores * 4, n, done.view(-1), 3)


@pytest.mark.parametrize("V,dtype", [(1 << 19, torch.float32), (1 << 20, torch.bfloat16), ((1 << 18) + 513, torch.float32)])
@pytest.mark.parametrize("K,alive", [(64, 0), (64, 63), (32, 7)])
def test_the_first_step_of_a_wide_group(K, alive, V, dtype):
    """One beam is alive, so that fewer threads than results hold anything."""
    logits, scores = _logits(1, K, V, V + K, dtype)
    scores = torch.full_like(scores, -math.inf)
    scores[0, alive] = -0.5
    _check(logits, scores, 64)
    up = torch.linspace(-9, 9, V, device="cuda").to(dtype)
    logits[alive] = up
    _check(logits, scores, 64)
    logits[alive] = up.flip(0)
    _check(logits, scores, 64)


@pytest.mark.parametrize("K,V,dtype", [(64, 131072, torch.bfloat16), (32, 131072, torch.float32)])
def test_wide_groups_are_not_gone_through_step_by_step(K, V, dtype):
    """Beams far apart cost no more than five times what beams side by side do (it was a hundred)."""
    logits, scores = _logits(4, K, V, K, dtype)

    def least(c):
        times = []
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            m.smla_beam_select(logits, c, 64)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    assert least(scores * 4) < 5 * least(scores * 0.05)
