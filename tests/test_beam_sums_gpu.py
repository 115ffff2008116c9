"""How far smla_beam_select's logarithm of a beam's sum may be off, which moves all of the beam's values.

A term e^d, d = x - maximum <= 0: d and its product with log2(e) are off by 2^-24 of d each, the exponential
by 2^-22 of its value.  A sum is brought to a new maximum at most once a step of its run (64) and once a run
that a lane goes through (16 with runs that long: 2^24 logits are 512 runs of 64 steps), and once more when the
lanes meet: 82 exponentials at most, 82 products, and d in parts whose sum is d.  Beside them 100 additions: 10
within a step, 80 of steps and runs, 10 between lanes.  The weighted mean of -d is ln V at most (the entropy of V
weights is ln V at most, and exceeds the mean of -d by ln sum >= 0), 16.7 for 2^24.  Together
    83 * 2^-22 + 182 * 2^-24 + 16.7 * 2^-23 = 3.3e-5
of the sum, which is the error of its logarithm; that itself adds 2^-23 (log1p in 32 bits, below 0.35).  2^-14 is
twice that.

The error is read off a second call: with the first one's value negated as the score, the value that comes back
is small, and its rounding to 32 bits with it."""
import pytest
import torch

import sparse_mla_decode_03_gb300 as m

pytestmark = pytest.mark.gpu
BOUND = 2.0 ** -14


def _check(x):
    first = m.smla_beam_select(x, torch.zeros(x.shape[0], 1, device="cuda"), 1)[2]
    rest = m.smla_beam_select(x, -first, 1)[2].double()
    d = x.double()
    want = -torch.logsumexp(d - d.amax(1, keepdim=True), 1, keepdim=True)
    off = (rest + first.double() - want).abs().max().item()
    assert off <= BOUND + 2.0 ** -24 * BOUND, f"off by {off:.3g}"


@pytest.mark.parametrize("V", [1000, 131072, 1 << 20, 1 << 24])
def test_normal_and_uniform_logits(V):
    g = torch.Generator(device="cuda").manual_seed(V)
    rows = max(2, min(64, (1 << 25) // V))
    for spread in (0.5, 2.0, 5.0):
        _check(torch.randn(rows, V, generator=g, device="cuda") * spread)
    _check((torch.randn(rows, V, generator=g, device="cuda") * 2).bfloat16())
    _check(torch.rand(rows, V, generator=g, device="cuda"))


@pytest.mark.parametrize("V", [1000, 131072, 1 << 20, 1 << 24])
@pytest.mark.parametrize("rows", [1, 4])
def test_sums_that_are_brought_to_a_new_maximum_with_every_step(V, rows):
    for height in (1e-3, 0.1, 9.0, 80.0):
        up = torch.linspace(-height, height, V, device="cuda").repeat(rows, 1)
        _check(up)
        _check(up.flip(1).contiguous())


@pytest.mark.parametrize("V", [1000, 131072, 1 << 24])
def test_equal_logits_and_one_ahead(V):
    x = torch.full((2, V), 1.5, device="cuda")
    _check(x)
    for ahead in (1e-3, 3.7, 20.0):
        x[:, V // 2] = 1.5 + ahead
        _check(x)
