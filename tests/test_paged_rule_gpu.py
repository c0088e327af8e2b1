"""Single tokens through both sets of kernels (the one-pass kernel and the block kernels)."""
import pytest
import torch

from tests import paged_cases as pc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("G", [1, 2, 4])
@pytest.mark.parametrize("width", [64, 2048, 16384])
def test_single_tokens_on_both_sides_of_the_rule(lib, d, fox, G, width):
    """Single tokens alone, with tables of 2^10, 2^15 and 2^18 positions a sequence: the kernels are
    chosen by what the tables could hold, the lengths stay short. Lengths at the borders of a key
    tile among them."""
    x = pc.make([0, 257, 128, 900], [1, 1, 1, 0], 2 * G, 2, d, 16, torch.bfloat16, fox, seed=44, width=width)
    before = pc.snapshot(x)
    out = pc.step(lib, x)
    pc.check(x, before, out)
