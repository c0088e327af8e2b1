"""How near bf16 steps behind a prefix come to 64 bits, by the roundings that their ways have.

With r = 1.53e-3 of the norm for one rounding to bf16 (half a step, 2^-8 over the significand, whose
mean square is 3 / (2 ln 2): 2^-8 / sqrt(3) / 1.47), a row whose weight lies with the prefix's keys has
  by one row tile          the output, the weights                            sqrt(2) r    = 2.17e-3
  by two at d = 64         the output (the weights have a second part)        r            = 1.53e-3
  by two at d = 128        output, query, half of the weights                 sqrt(2.5) r  = 2.42e-3
  all three                                                                   sqrt(3) r    = 2.65e-3
The bar lies between the last two, 2.5e-3: chunks whose queries are rounded once and their weights
too would be above it."""
import pytest
import torch

from tests import paged_prefix_cases as px

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("members,T", [(40, 1), (8, 7), (40, 7), (4, 64), (4, 65), (3, 130), (2, 300)])
def test_behind_a_long_prefix(lib, d, fox, members, T):
    x = px.make([4000] + [20] * members, [0] + [T] * members, [-1] + [0] * members, 8, 2, d, 64, torch.bfloat16,
                fox, seed=61)
    ref = px.reference(x)[0]
    out = px.step(lib, x)
    assert float((out.double() - ref).norm() / ref.norm()) <= 2.5e-3
