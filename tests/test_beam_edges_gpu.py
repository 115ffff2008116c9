"""smla_beam_select where many candidates are equal, against the definition in 64 bits (tolerances:
_rows4_helpers).  Sums are whole numbers here, and powers of two, so that ties are exact."""
import math

import pytest
import torch

from test_beam_gpu import _check

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
