"""How near bf16 steps come to 64 bits: bounds by the number of roundings to bf16 that a way through
the kernels has, closer than those that the other tests use.

One rounding to bf16 is off by at most half a step, 2^-8 of the value over its significand s in [1, 2),
evenly within that: 2^-8 / sqrt(3) / s (root mean square), and with significands spread evenly in
their logarithm (mean square of s: 3 / (2 ln 2) = 2.16) r = 2^-8 / sqrt(3) / 1.47 = 1.53e-3 of the
norm. Roundings of an output, of softmax weights and of a carried query (whose logits are of unit size)
each add r^2 to the squared error, weights with a second part for half of the keys half of that:
  one-pass kernel          the output                                  r            = 1.53e-3
  with cached keys         the output, the weights                     sqrt(2) r    = 2.17e-3
  long chunks at d = 128   and the carried query, half of the weights  sqrt(2.5) r  = 2.42e-3
  one part more left out                                               sqrt(3) r    = 2.65e-3
The bars lie between what a case has and one rounding more: 1.85e-3 (between r and sqrt(2) r) and
2.5e-3 (between sqrt(2.5) r and sqrt(3) r)."""
import pytest
import torch

from tests import paged_cases as pc

pytestmark = pytest.mark.gpu


def error(lib, x):
    ref = pc.reference(x)[0]
    out = pc.step(lib, x)
    return float((out.double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("n,T", [(0, 300), (1000, 300)])
def test_chunks_of_several_blocks(lib, d, fox, n, T):
    x = pc.make([n], [T], 4, 4, d, 64, torch.bfloat16, fox, seed=51)
    assert error(lib, x) <= 2.5e-3


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("Hq,Hkv,T,bar", [
    (8, 8, 1, 1.85e-3),    # one pass
    (12, 4, 1, 2.5e-3),    # the block kernels, one row tile a key head
    (8, 4, 7, 2.5e-3),
])
def test_few_tokens_over_a_cache(lib, d, fox, Hq, Hkv, T, bar):
    x = pc.make([1000 + 37 * s for s in range(8)], [T] * 8, Hq, Hkv, d, 16, torch.bfloat16, fox, seed=52)
    assert error(lib, x) <= bar
