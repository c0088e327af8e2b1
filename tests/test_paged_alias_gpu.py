"""Steps whose output takes the place of an input."""
import pytest
import torch

from tests import paged_cases as pc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fox", [False, True])
@pytest.mark.parametrize("chunks", [[1, 1, 1], [5, 0, 1], [1, 150, 1]])
@pytest.mark.parametrize("Hq,name", [(2, "q"), (2, "k"), (2, "v"), (2, "w"), (6, "q")])
def test_out_in_the_place_of_an_input(lib, dtype, fox, chunks, Hq, name):
    x = pc.make([300, 20, 0], chunks, Hq, 2, 64, 16, dtype, fox, seed=61)
    y = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    before = pc.snapshot(x)
    out = pc.step(lib, x)
    pc.check(x, before, out)
    assert torch.equal(pc.step(lib, y, out=y[name]), out)
    for n in before:
        if x[n] is not None:
            assert torch.equal(x[n].nan_to_num(nan=7.0), y[n].nan_to_num(nan=7.0))
