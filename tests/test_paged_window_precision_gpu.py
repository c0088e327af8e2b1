"""How near bf16 steps through a window come to 64 bits, by the roundings that their ways have: with
r = 1.53e-3 of the norm for one rounding to bf16 (2^-8 / sqrt(3) over a significand of 1.47, root mean
square), the output and the weights sqrt(2) r = 2.17e-3; in chunks at d = 128 the output, the query and a
quarter of the weights sqrt(2.25) r = 2.30e-3; the output, the query and all weights sqrt(3) r = 2.65e-3.
The bar lies between the last two, nearer to the first: 2.45e-3."""
import pytest
import torch

from tests import paged_cases as pc
from tests import paged_window_cases as wc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("seqs,T", [(40, 1), (6, 7), (4, 64), (4, 65), (2, 100)])
def test_through_a_long_window(lib, d, fox, seqs, T):
    x = pc.make([9000] * seqs, [T] * seqs, 8, 2, d, 64, torch.bfloat16, fox, seed=71)
    ref = wc.window_reference(x, 8000, 4)[0]
    out = wc.window_step(lib, x, pc.cache_of(lib, x), 8000, 4)
    assert float((out.double() - ref).norm() / ref.norm()) <= 2.45e-3
